// qmm_q8c.cuh -- 8-bit products with one scale per output channel and one per
// activation row (token): the laid-out weights and what the row kernel
// (qmm_q8c_rows.cu) and the tcgen05 GEMM (qmm_q8c_gemm.cu) share.
//
//   y[m][n] = (sum_k a[m][k] w[n][k]) sw[n] sx[m] (+ bias[n]),  a, w in -128..127
//
// The pages pair Q8_0 weights with activations that are quantized per row in
// blocks of 32 ("同一个 GGUF…" section 出处); here a whole row is one block,
// the rule for its scale and codes is the same (d = max|x| / 127, "自己量化"
// section 和下载的 Q8_0 逐字节比).
//
// Every path forms the integer sum exactly, whatever its order, and scales it
// in the same way, so that a row's result depends neither on the kernel nor on
// the other rows of the call.
//
// Laid out, the weights are row blocks of 16 rows in segments of 128 K, 2 KB
// each: two tiles of 64 K, of which 512 bytes are rows 0..7 and 512 rows 8..15,
// lane l = 4 g + t of a warp holding K 16 t .. 16 t + 15 of row g (g + 8) at byte
// 16 l.  Eight row blocks are a panel, whose segments of the same K are next to
// each other, 16 KB that the GEMM copies in one piece (a box of eight 2 KB pieces
// took the copy engine 590 ns, more than the rest of a tile takes); the last
// panel has as many row blocks as there are.  A lane's two 16-byte loads are its operands of two
// m16n8k32 integer MMAs (words 2 i, 2 i + 1 of MMA i; the activations' words in
// the same order) and, turned into f16, of a 16-lane x 128-bit tensor-memory
// store.  Rows past N and K past the row's end are 0.  Behind the row blocks:
// f32 scales of their rows, and the largest sum of squares of a row's codes.
#pragma once

#include "qmm_internal.h"
#include "qmm_q4g.cuh"

namespace qmm {

constexpr int kQcSeg = 2048;  // bytes of a segment: 16 rows x 128 K
constexpr int kQcMaxK = (1 << 17) - 1;  // |sum| <= K 2^14 < 2^31

struct QcWeights {
    const uint8_t* data;
    int N, K;
    int RB, KS;            // row blocks, segments per row block
    long long scale_off;   // bytes to the scales, f32 [RB * 16]
    long long norm_off;    // bytes to the largest sum of squares, u32
};

inline bool qc_describe(long long N, long long K, const void* data, QcWeights& w) {
    if (N < 1 || K < 1 || N > (1 << 23) || K > kQcMaxK) return false;
    w.data = static_cast<const uint8_t*>(data);
    w.N = (int)N;
    w.K = (int)K;
    w.RB = (int)((N + 15) / 16);
    w.KS = (int)((K + 127) / 128);
    w.scale_off = (long long)w.RB * w.KS * kQcSeg;
    w.norm_off = w.scale_off + (long long)w.RB * 64;
    return true;
}
// a row block's first segment, and the bytes from a segment to the next
__host__ __device__ inline long long qc_row_block(const QcWeights& w, int rb) { return ((long long)(rb & ~7) * w.KS + (rb & 7)) * kQcSeg; }
__host__ __device__ inline int qc_step(const QcWeights& w, int rb) { return (w.RB - (rb & ~7) < 8 ? w.RB - (rb & ~7) : 8) * kQcSeg; }
inline size_t qc_bytes(const QcWeights& w) { return (size_t)w.norm_off + 16; }

// Activations of a call: floats, quantized on the way, or codes with a scale per row.  Kernels read them, and what
// an earlier launch of the call made, by plain loads: __ldg is for data that nobody writes while the kernel runs, and a
// kernel that was started early runs while the grid before it writes.  (By __ldcg every block asks L2 for the same
// scales: 64 x 4096 x 4096 14.5 us, with plain loads 13.2.)
struct QcRows {
    const void* x;        // float rows (xt), or int8 codes (scales given)
    const float* scales;  // NULL: x is float
    long long ld;         // elements from a row to the next
    int xt;
    int M;
};
struct QcCall {
    QcWeights w;
    QcRows a;
    const float* bias;
    void* y;
    int yt;
};

// one result from its integer sum (as the nearest float), the same on every path
__device__ __forceinline__ float qc_scale(float sum, float sw, float sx, float bias) {
    return __fadd_rn(__fmul_rn(__fmul_rn(sum, sw), sx), bias);
}

// The scale of a row from the bits of its largest magnitude (an infinity's or a NaN's are above every
// number's): d, and the reciprocal that its values are multiplied by.  A row that is not finite has
// scale NaN and codes 0, so that its results are NaN.
__device__ __forceinline__ void qc_row_scale(uint32_t top, float& d, float& id) {
    q8_scale(__uint_as_float(top), d, id);
    if (top >= 0x7f800000u) {
        d = __uint_as_float(0x7fc00000u);
        id = 0.0f;
    }
}
__device__ __forceinline__ uint32_t qc_abs_bits(float v) { return __float_as_uint(v) & 0x7fffffffu; }

// Four words of f16 or bf16 pairs as floats.
template <int XT>
__device__ __forceinline__ void qc_words8(const uint32_t w[4], float f[8]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if constexpr (XT == X_F16) {
            const float2 v = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
            f[2 * i] = v.x;
            f[2 * i + 1] = v.y;
        } else {
            f[2 * i] = __uint_as_float(w[i] << 16);
            f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
        }
    }
}
// Eight consecutive values of a row on 16-byte boundaries, from element k, as floats.
template <int XT>
__device__ __forceinline__ void qc_row8(const void* row, int k, float f[8]) {
    if constexpr (XT == X_F32) {
        const float4 a = *reinterpret_cast<const float4*>(static_cast<const float*>(row) + k);
        const float4 b = *(reinterpret_cast<const float4*>(static_cast<const float*>(row) + k) + 1);
        f[0] = a.x, f[1] = a.y, f[2] = a.z, f[3] = a.w, f[4] = b.x, f[5] = b.y, f[6] = b.z, f[7] = b.w;
    } else {
        const uint4 u = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(row) + k);
        const uint32_t w[4] = {u.x, u.y, u.z, u.w};
        qc_words8<XT>(w, f);
    }
}
// The same of any row (vec: it is on 16-byte boundaries), 0 from K on.
template <int XT>
__device__ __forceinline__ void qc_load8(const void* row, int k, int K, bool vec, float f[8]) {
    if (vec && k + 8 <= K) {
        qc_row8<XT>(row, k, f);
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) f[i] = k + i < K ? x_load(row, XT, k + i) : 0.0f;
    }
}
// v = x id in -128..128: the sum v + 1.5 2^23 has its nearest integer (ties to even) in the low byte; a
// tie that went towards zero is put right, so that halves go away from zero, as in q8_code.
__device__ __forceinline__ uint32_t qc_code_word(float x, float id) {
    const float magic = 12582912.0f, v = __fmul_rn(x, id);
    float sum = __fadd_rn(v, magic);
    const float rest = __fsub_rn(v, __fsub_rn(sum, magic)), half = __uint_as_float((__float_as_uint(v) & 0x80000000u) | 0x3f000000u);
    if (rest == half) sum = __fadd_rn(sum, __fadd_rn(half, half));
    return __float_as_uint(sum);
}
// Eight codes.  A reciprocal that overflowed, or 0 (a row of zeros, or one that is not finite), takes the long
// way, where a product may be infinite or NaN.
__device__ __forceinline__ uint2 qc_codes8(const float f[8], float id) {
    if (id > 1e38f || id == 0.0f)
        return make_uint2(pack4(q8_code(f[0], id), q8_code(f[1], id), q8_code(f[2], id), q8_code(f[3], id)),
                          pack4(q8_code(f[4], id), q8_code(f[5], id), q8_code(f[6], id), q8_code(f[7], id)));
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = __byte_perm(qc_code_word(f[2 * i], id), qc_code_word(f[2 * i + 1], id), 0x0040u);
    return make_uint2(__byte_perm(w[0], w[1], 0x5410u), __byte_perm(w[2], w[3], 0x5410u));
}

// Four signed bytes as two f16 pairs, exact.
__device__ __forceinline__ void qc_half4(uint32_t w, uint32_t& lo, uint32_t& hi) {
    const __half2 bias = __half2(__ushort_as_half(0x6480), __ushort_as_half(0x6480));  // 1152
    const uint32_t u = w ^ 0x80808080u;
    uint32_t a = __byte_perm(u, 0x64646464u, SEL01), b = __byte_perm(u, 0x64646464u, SEL23);  // 1024 + 128 + q
    const __half2 ra = __hsub2(*reinterpret_cast<__half2*>(&a), bias), rb = __hsub2(*reinterpret_cast<__half2*>(&b), bias);
    lo = *reinterpret_cast<const uint32_t*>(&ra);
    hi = *reinterpret_cast<const uint32_t*>(&rb);
}

cudaError_t launch_q8c_pack(const int8_t* codes, long long ldc, const float* scales, const QcWeights& w, void* out, cudaStream_t s);
cudaError_t launch_q8c_dequantize(const QcWeights& w, float* out, cudaStream_t s);
cudaError_t launch_q8c_quantize(const QcRows& a, int K, int8_t* codes, long long ldc, float* scales, cudaStream_t s);

// The preparation of a call's activations.  f16: codes as f16, rows of 64-K tiles in the order of the
// laid-out weights' lanes, and the sums of squares; else int8 codes, rows of `pitch` bytes.  Zeros
// fill a row up to the pitch.
struct QcPrep {
    void* codes;
    float* scales;
    uint32_t* norms;  // f16
    long long pitch;  // elements
};
cudaError_t launch_q8c_prep(const QcRows& a, int K, const QcPrep& p, bool f16, cudaStream_t s);

struct QcRowsPlan {
    bool ok = false;
    int warps = 0, blocks = 0;
    int pitch = 0;       // bytes of a staged row
    int prep = 0;        // activations are quantized (or aligned) by a launch of their own
    int off_zero = 0, off_part = 0, off_ring = 0;
    size_t smem = 0, workspace = 0;
};
QcRowsPlan plan_q8c_rows(const QcCall& c, int sms, int smem_max);
cudaError_t launch_q8c_rows(const QcRowsPlan& pl, const QcCall& c, void* ws, int smem_max, cudaStream_t s);

struct QcGemmPlan {
    bool ok = false;
    int cg = 0, kt = 0, bx = 0, nacc = 0, accw = 0, mtiles = 0, ntiles = 0, nraw = 0, nx = 0, nstage = 0, grid = 0, ks = 0;
    size_t smem = 0, ws_scale = 0, ws_norm = 0, ws_part = 0, workspace = 0;
};
QcGemmPlan plan_q8c_gemm(const QcCall& c, int sms, int smem_max);
// Whether 16-bit results may be stored four neighbours of a row at a time, 8 bytes: y itself is aligned only as its
// elements are, and rows follow each other without a gap.
inline bool qc_wide_results(const QcCall& c, int ks) {
    return c.yt != X_F32 && ks == 1 && c.w.N % 4 == 0 && (reinterpret_cast<uintptr_t>(c.y) & 7) == 0;
}
cudaError_t launch_q8c_gemm(const QcGemmPlan& pl, const QcCall& c, void* ws, unsigned* err, int stall, int smem_max, cudaStream_t s);

// Norms around a block; see include/qmm.h (qmm_block_norm).
struct NormCall {
    const void *y, *r, *gate, *post, *pre;
    void *r_out, *h;      // h: float result, or NULL
    int8_t* codes;        // or codes and scales
    float* scales;
    long long ldy, ldr, ldg, ldro, ldh;
    int T, K, xt, wt;
    float scale, eps, offset;
};
struct NormParams {
    NormCall c;
    int vec;  // every row, and every one of its 8-value pieces, starts on its natural boundary
};
cudaError_t launch_block_norm(const NormCall& c, cudaStream_t s);
cudaError_t launch_block_norm_f32(const NormParams& p, cudaStream_t s);
cudaError_t launch_block_norm_f16(const NormParams& p, cudaStream_t s);
cudaError_t launch_block_norm_bf16(const NormParams& p, cudaStream_t s);

}  // namespace qmm
