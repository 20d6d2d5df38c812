// qmm_q4g.cuh -- 4-bit weights with group scales: the laid-out form that the
// row kernel (qmm_q4g_rows.cuh) and the tcgen05 GEMM (qmm_q4g_gemm.cuh) read.
//
//   w[n][k] = s[n][k / G] (q[n][k] - z[n][k / G]),  q, z in 0..15, G = 32, 64 or 128
//
// The pages quantize weights row by row in blocks along K ("自己量化" section
// 3, QTensor::quantize); this is that form with the scales beside the codes
// and a zero point per group (Q4_0 is the case G = 32, z = 8).
//
// Laid out, a weight matrix is row blocks of 16 rows, each one contiguous
// stream of segments of 128 K:
//   segment: 2 tiles of 512 B (16 rows x 64 K codes), then 16 rows x 128 / G
//            scale words
//   tile:    lane l = 4 g + t of a warp holds one uint4: word s has the codes
//            of the 16-K step s in the A-fragment order of the 16 x 16 warp
//            MMA, which is also the order of a 16-lane x 128-bit tensor-memory
//            store: nibble i (0..3) is the low and nibble i + 4 the high half
//            of fragment register i: registers 0, 1: rows g, g + 8, K = 16 s +
//            2 t, + 1; registers 2, 3: the same rows, K + 8
//   scales:  [g][group][2]: rows g and g + 8; a word is the f32 scale with the
//            zero point in its low 4 bits (f16 and bf16 scales have at most 11
//            significant bits, so those 13 bits of the f32 are zero: exact)
// so one coalesced 512-byte load per warp is a whole MMA operand, and 8 row
// blocks of a segment are a GEMM tile's raw stage.  Rows past N and K past the
// row's end have scale 0.  In a paired matrix (an expert's gate and up rows,
// N = 2 F) block b holds gate rows 8 b.. as rows 0..7 and up rows 8 b.. as
// rows 8..15, so that a thread that has a gate row's sum has its up row's too.
// After the last expert come f32 powers of two, one per row in layout order:
// 2^-e with max_g 15 |s| 2^e in [2^14, 2^15), the scale that brings a row's
// weights into f16's range for the GEMM.
#pragma once

#include <cuda_bf16.h>

#include "qmm_device.cuh"

namespace qmm {

enum : int { X_F32 = 0, X_F16 = 1, X_BF16 = 2 };  // activation and output types
__host__ __device__ constexpr int x_size(int xt) { return xt == X_F32 ? 4 : 2; }

constexpr int kQgRows = 16;    // rows per row block
constexpr int kQgSegK = 128;   // K per segment
constexpr int kQgTile = 512;   // bytes of a tile's codes
__host__ __device__ constexpr int qg_seg_bytes(int ng) { return 2 * kQgTile + 64 * ng; }  // ng = 128 / G scale words a row

// A laid-out weight matrix.
struct QgWeights {
    const uint8_t* data;
    long long expert_stride;  // bytes from an expert to the next
    long long iscale_off;     // bytes to the row powers of two, f32 [E][RB * 16]
    int E, N, K;
    int RB, KS;               // row blocks, segments per row block
    int ng;                   // scale words per row and segment: 1, 2, 4
    int paired;
};

inline bool qg_describe(long long E, long long N, long long K, int group, int paired, const void* data, QgWeights& w) {
    if (E < 1 || N < 1 || K < 1 || E > 65535 || N > (1 << 23) || K > (1 << 20)) return false;
    if (group < 32 || group % 32 != 0 || K % group != 0 || (paired && N % 2 != 0)) return false;
    w.data = static_cast<const uint8_t*>(data);
    w.E = (int)E;
    w.N = (int)N;
    w.K = (int)K;
    w.paired = paired ? 1 : 0;
    w.RB = paired ? (int)((N / 2 + 7) / 8) : (int)((N + 15) / 16);
    w.KS = (int)((K + kQgSegK - 1) / kQgSegK);
    w.ng = group % 128 == 0 ? 1 : group % 64 == 0 ? 2 : 4;
    w.expert_stride = (long long)w.RB * w.KS * qg_seg_bytes(w.ng);
    w.iscale_off = w.expert_stride * E;
    return true;
}

// the weight row that layout row r (0..15) of row block rb holds; -1: none
__host__ __device__ inline int qg_row(const QgWeights& w, int rb, int r) {
    if (w.paired) {
        const int f = rb * 8 + (r & 7), F = w.N / 2;
        return f < F ? (r < 8 ? f : F + f) : -1;
    }
    const int n = rb * 16 + r;
    return n < w.N ? n : -1;
}

__device__ __forceinline__ float qg_scale(uint32_t sw) { return __uint_as_float(sw & ~15u); }

__device__ __forceinline__ float x_load(const void* p, int xt, long long i) {
    if (xt == X_F32) return static_cast<const float*>(p)[i];
    if (xt == X_F16) return __half2float(static_cast<const __half*>(p)[i]);
    return __bfloat162float(static_cast<const __nv_bfloat16*>(p)[i]);
}
__device__ __forceinline__ void x_store(void* p, int xt, long long i, float v) {
    if (xt == X_F32) static_cast<float*>(p)[i] = v;
    else if (xt == X_F16) static_cast<__half*>(p)[i] = __float2half_rn(v);
    else static_cast<__nv_bfloat16*>(p)[i] = __float2bfloat16_rn(v);
}

// Bounded wait whose tries suspend the warp (for up to 2 us each) instead of
// returning at once: 20 waiting warps that spin take a third of the issue slots
// that the converting ones need.
__device__ __forceinline__ bool qg_wait(uint32_t bar, uint32_t parity, volatile int* abort_flag, unsigned* err) {
    if (mbar_try(bar, parity)) return true;
    const long long t0 = clock64();
    while (true) {
        uint32_t ok;
        asm volatile(
            "{\n\t.reg .pred p;\n\tmbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n\tselp.u32 %0, 1, 0, p;\n\t}"
            : "=r"(ok)
            : "r"(bar), "r"(parity), "r"(2000u)
            : "memory");
        if (ok) return true;
        if (*abort_flag) return false;
        if (clock64() - t0 > kWaitLimitCheck) return mbar_spin(bar, parity, abort_flag, err, false);  // raises the error in the end
    }
}
// The same for a whole warp, with one answer for all of its lanes: each lane's own depends on its
// tries, clock and reading of the abort flag, and a warp that left its loop in part would wait
// without end at the next instruction that all lanes take part in.  ready: the phase was seen
// complete before.
__device__ __forceinline__ bool qg_wait_warp(uint32_t bar, uint32_t parity, bool ready, volatile int* abort_flag, unsigned* err) {
    return __all_sync(0xffffffffu, ready || qg_wait(bar, parity, abort_flag, err));
}

// A place in a ring of n stages: its index and the parity of its current use.
// A producer waits for a stage's release with ph ^ 1, which a fresh barrier
// passes.  (Counting uses and dividing by a run-time n costs the MMA thread
// more than its four MMAs.)
struct QgRing {
    int s = 0;
    uint32_t ph = 0;
    __device__ __forceinline__ void next(int n) {
        if (++s == n) {
            s = 0;
            ph ^= 1u;
        }
    }
    __device__ __forceinline__ void skip(int k, int n) {
        for (s += k; s >= n; s -= n) ph ^= 1u;
    }
};
template <typename Y>
__device__ __forceinline__ Y to_type(float v);
template <>
__device__ __forceinline__ float to_type<float>(float v) { return v; }
template <>
__device__ __forceinline__ __half to_type<__half>(float v) { return __float2half_rn(v); }
template <>
__device__ __forceinline__ __nv_bfloat16 to_type<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }

// silu(g) u; the fast form (a few units of 2^-22) where the result is rounded to 16 bits
__device__ __forceinline__ float swiglu_fast(float g, float u) { return __fdividef(g, 1.0f + __expf(-g)) * u; }
__device__ __forceinline__ float swiglu(float g, float u) { return g / (1.0f + expf(-g)) * u; }

}  // namespace qmm
