// qmm_norm.cuh -- what stands between two blocks of a decoder in one pass: the
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
// maximum).  Three kernels, in all of which a row is dealt to as many threads and
// summed in the same order, so that its results are the same bits beside
// any other rows:
//   block_norm_kernel, a block (short rows: a warp) per row: rows on no 16-byte boundaries, K past 8192, weights of
//     the other 16-bit type, few long rows; bound by a launch, one trip to memory and the reductions
//   norm_ring_kernel: persistent blocks, a row at a time, whose next rows are on their way into a ring in shared
//     memory by bulk copies; weights and a gate per channel stay in registers.  4096 rows of 4096 in bf16, norms on
//     both sides, a gate per channel: 24.7 us, 5.4 TB/s (a block per row: 46, loads and reductions in turn)
//   norm_warps_kernel: short rows, a warp each, the next one in registers; 16384 of 576 in f16 20.4 us
#pragma once

#include <type_traits>

#include "qmm_q8c.cuh"

namespace qmm {
namespace {

template <int XT>
__device__ __forceinline__ uint32_t two16(float a, float b) {
    if constexpr (XT == X_F16) {
        const __half2 v = __floats2half2_rn(a, b);
        return *reinterpret_cast<const uint32_t*>(&v);
    } else {
        const __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
        return *reinterpret_cast<const uint32_t*>(&v);
    }
}
template <int XT>
__device__ __forceinline__ void store8(void* row, int k, int K, const float f[8]) {
    if (k + 8 <= K) {
        if constexpr (XT == X_F32) {
            float4* p = reinterpret_cast<float4*>(static_cast<float*>(row) + k);
            p[0] = make_float4(f[0], f[1], f[2], f[3]);
            p[1] = make_float4(f[4], f[5], f[6], f[7]);
        } else {
            uint32_t w[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) w[i] = two16<XT>(f[2 * i], f[2 * i + 1]);
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

__device__ __forceinline__ float root_of(float ss, const NormCall& c) { return 1.0f / sqrtf(fmaf(ss, 1.0f / (float)c.K, c.eps)); }

// A thread's 8 neighbouring values of a row.  VEC: rows start on 16-byte boundaries; else a warp's pieces are taken
// from the 16-byte words that they lie in: a lane asks for the words that its piece begins in, has what it misses
// from the next lane (the last one: from memory) and shifts.  A word that is not in the tensor whole is read value
// by value; other words may hold neighbouring rows' values, which are dropped.  So a thread's values are the same
// wherever a row starts.  4096 rows of 4095 in bf16, a gate per token: 65 us (eight loads of a value each 122; 32
// values apart and exchanged through shared memory 98).
template <int XT, bool VEC>
struct Piece {
    static constexpr int kWords = XT == X_F32 ? 8 : 4, kEach = 16 / x_size(XT);  // 4-byte words; values of a 16-byte word
    uint32_t u[kWords + 4];
    int o;  // bytes from a 16-byte boundary to the piece, the same for a row

    // The 16-byte word from value k of a row on.  ENDS: only values lo .. hi - 1 from the row's start on are the
    // tensor's; then value by value, others in place of those that are not there.
    template <bool ENDS>
    static __device__ __forceinline__ void word(const uint8_t* row, int k, int lo, int hi, bool on, uint32_t* to) {
        to[0] = to[1] = to[2] = to[3] = 0u;
        if (!on) return;
        if constexpr (!ENDS) {
            const uint4 v = *reinterpret_cast<const uint4*>(row + k * x_size(XT));
            to[0] = v.x, to[1] = v.y, to[2] = v.z, to[3] = v.w;
        } else {
            auto one = [&](int e) {
                const int i = max(min(k + e, hi - 1), lo);
                if constexpr (XT == X_F32) return reinterpret_cast<const uint32_t*>(row)[i];
                else return (uint32_t)reinterpret_cast<const uint16_t*>(row)[i];
            };
#pragma unroll
            for (int i = 0; i < 4; ++i) to[i] = XT == X_F32 ? one(i) : one(2 * i) | one(2 * i + 1) << 16;
        }
    }
    // values k .. k + 7: the words that begin in the row
    template <bool ENDS>
    __device__ __forceinline__ void load(const void* from, int k, int lo, int hi, int K) {
        const uint8_t* row = static_cast<const uint8_t*>(from);
        if constexpr (!VEC) o = (int)(reinterpret_cast<uintptr_t>(row) & 15);
        const int k0 = k - (VEC ? 0 : o / x_size(XT));
#pragma unroll
        for (int i = 0; i < kWords; i += 4) word<ENDS>(row, k0 + i / 4 * kEach, lo, hi, k0 + i / 4 * kEach < K, u + i);
        if constexpr (!VEC) word<ENDS>(row, k0 + 8, lo, hi, (threadIdx.x & 31) == 31 && o && k0 + 8 < K, u + kWords);
    }
    // Whether the words of a warp's 256 values, this lane's from k on, may lie in the tensor in part: at most 7 values
    // before and after the row are read.
    static __device__ __forceinline__ bool ends(bool first, bool last, int k, int K) {
        if (VEC && K % 8 == 0) return false;
        k -= 8 * (threadIdx.x & 31);
        return (first && k == 0) || (last && k + 256 + 8 > K);
    }
    // of a row that is a tensor
    __device__ __forceinline__ void load_one(const void* row, int k, int K) {
        if (ends((reinterpret_cast<uintptr_t>(row) & 15) != 0, true, k, K)) load<true>(row, k, 0, K, K);
        else load<false>(row, k, 0, K, K);
    }
    // n words of w from `bytes` (< 16) on
    template <int N>
    static __device__ __forceinline__ void shift(uint32_t* w, int bytes) {
#pragma unroll
        for (int i = 0; i < N + 2; ++i) w[i] = bytes & 8 ? w[i + 2] : w[i];
#pragma unroll
        for (int i = 0; i < N + 1; ++i) w[i] = bytes & 4 ? w[i + 1] : w[i];
        if constexpr (XT != X_F32) {
#pragma unroll
            for (int i = 0; i < N; ++i) w[i] = __funnelshift_r(w[i], w[i + 1], 8 * (bytes & 2));
        }
    }
    // 0 from K on
    __device__ __forceinline__ void get(int k, int K, float f[8]) {
        if constexpr (!VEC) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const uint32_t next = __shfl_down_sync(0xffffffffu, u[i], 1);
                if ((threadIdx.x & 31) != 31) u[kWords + i] = next;
            }
            shift<kWords>(u, o);
        }
        if constexpr (XT == X_F32) {
#pragma unroll
            for (int i = 0; i < 8; ++i) f[i] = __uint_as_float(u[i]);
        } else {
            qc_words8<XT>(u, f);
        }
        if (k + 8 > K) {
#pragma unroll
            for (int e = 0; e < 8; ++e) f[e] = k + e < K ? f[e] : 0.0f;
        }
    }
    // values to the row, likewise in whole words but for a warp's ends and the row's
    __device__ __forceinline__ void store(void* p, int k, int K, const float f[8]) {
        if constexpr (VEC) {
            store8<XT>(p, k, K, f);
            return;
        }
        uint8_t* row = static_cast<uint8_t*>(p);
        const int lane = threadIdx.x & 31, from = (16 - (int)(reinterpret_cast<uintptr_t>(row) & 15)) & 15, head = from / x_size(XT);
        if constexpr (XT == X_F32) {
#pragma unroll
            for (int i = 0; i < 8; ++i) u[i] = __float_as_uint(f[i]);
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i) u[i] = two16<XT>(f[2 * i], f[2 * i + 1]);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) u[kWords + i] = __shfl_down_sync(0xffffffffu, u[i], 1);
        shift<kWords>(u, from);
        // values head .. 7 of this piece and 0 .. head - 1 of the next one are the words; the first `head` are the last lane's
        const bool before = head && lane > 0 && k + head <= K;
        int done = head;  // values up to here are in words
#pragma unroll
        for (int i = 0; i < kWords; i += 4) {
            const int k1 = k + head + i / 4 * kEach;
            if (k1 + kEach <= K && (i + 4 < kWords || head == 0 || lane < 31)) {
                *reinterpret_cast<uint4*>(row + (long long)k1 * x_size(XT)) = make_uint4(u[i], u[i + 1], u[i + 2], u[i + 3]);
                done = head + (i / 4 + 1) * kEach;
            }
        }
#pragma unroll
        for (int e = 0; e < 8; ++e)
            if (k + e < K && (e < head ? !before : e >= done)) x_store(row, XT, k + e, f[e]);
    }
};

// Piece j of a row of y (Y), of residual and gate (RG).  The first and the last row of a tensor have its ends.
template <bool Y, bool RG, int XT, bool VEC, int TPR>
__device__ __forceinline__ void load_piece(const NormCall& c, long long row, int lane, int j, Piece<XT, VEC>& y, Piece<XT, VEC>& r, Piece<XT, VEC>& gate) {
    const int before = (int)min(row * c.K, 8ll), after = (int)min((c.T - 1 - row) * c.K, 8ll), k = 8 * (lane + TPR * j);
    auto at = [&](const void* base, long long ld) { return static_cast<const uint8_t*>(base) + row * ld * x_size(XT); };
    auto load = [&](auto ends) {
        constexpr bool kEnds = decltype(ends)::value;
        if (Y) y.template load<kEnds>(at(c.y, c.ldy), k, -before, c.K + after, c.K);
        if (RG && c.r) r.template load<kEnds>(at(c.r, c.ldr), k, -before, c.K + after, c.K);
        if (RG && c.gate && c.ldg) gate.template load<kEnds>(at(c.gate, c.ldg), k, -before, c.K + after, c.K);
    };
    if (Piece<XT, VEC>::ends(before < 8, after < 8, k, c.K)) load(std::true_type());
    else load(std::false_type());
    if (RG && c.gate && !c.ldg) gate.load_one(c.gate, k, c.K);  // for all rows
}
template <int XT, bool VEC, int TPR, int NV>
__device__ __forceinline__ void store_row(void* row, int lane, int K, const float f[NV][8]) {
#pragma unroll
    for (int j = 0; j < NV; ++j) {
        Piece<XT, VEC> p;
        p.store(row, 8 * (lane + TPR * j), K, f[j]);
    }
}
template <int WT, bool VEC>
__device__ __forceinline__ void weight_piece(const void* weight, int k, int K, float f[8]) {
    Piece<WT, VEC> p;
    p.load_one(weight, k, K);
    p.get(k, K, f);
}
// v = v root (offset + weight)
template <bool VEC, int TPR, int NV>
__device__ __forceinline__ void weigh(const NormCall& c, const void* weight, float root, int lane, float v[NV][8]) {
#pragma unroll
    for (int j = 0; j < NV; ++j) {
        float w[8];
        const int k = 8 * (lane + TPR * j);
        if (c.wt == X_F32) weight_piece<X_F32, VEC>(weight, k, c.K, w);
        else if (c.wt == X_F16) weight_piece<X_F16, VEC>(weight, k, c.K, w);
        else weight_piece<X_BF16, VEC>(weight, k, c.K, w);
#pragma unroll
        for (int e = 0; e < 8; ++e) v[j][e] = v[j][e] * root * (c.offset + w[e]);
    }
}

// TPR threads and NV pieces a row, as in the kernels for many rows, and the same operations in the same order:
// a row's results depend neither on the kernel nor on the other rows.
template <int XT, int TPR, int NV, bool VEC>
__global__ void __launch_bounds__(TPR == 32 ? 64 : TPR) block_norm_kernel(const NormParams p) {
    constexpr int kRows = TPR == 32 ? 2 : 1;
    __shared__ float red[3][32];  // an area per reduction
    grid_dep_launch();
    const NormCall& c = p.c;
    const int lane = threadIdx.x % TPR, K = c.K;
    const long long row = (long long)blockIdx.x * kRows + threadIdx.x / TPR;
    grid_dep_wait();
    if (row >= c.T) return;  // whole warps; blocks of one row have theirs
    constexpr bool kLate = NV > 3;  // residual and gate where they are used, as registers do not hold them (rows of 14336 in bf16 as four pieces 8.2 us, with all at once 12)
    Piece<XT, VEC> y[NV], r[NV], gate[NV];
    float v[NV][8];
#pragma unroll
    for (int j = 0; j < NV; ++j) load_piece<true, !kLate, XT, VEC, TPR>(c, row, lane, j, y[j], r[j], gate[j]);
#pragma unroll
    for (int j = 0; j < NV; ++j) y[j].get(8 * (lane + TPR * j), K, v[j]);
    if (c.post) {
        float s0 = 0.0f, s1 = 0.0f;
#pragma unroll
        for (int j = 0; j < NV; ++j)
#pragma unroll
            for (int e = 0; e < 8; e += 2) {
                s0 = fmaf(v[j][e], v[j][e], s0);
                s1 = fmaf(v[j][e + 1], v[j][e + 1], s1);
            }
        weigh<VEC, TPR, NV>(c, c.post, root_of(sum_row<TPR>(s0 + s1, red[0]), c), lane, v);
    }
    float s0 = 0.0f, s1 = 0.0f;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
        float f[8];
        if (kLate) load_piece<false, true, XT, VEC, TPR>(c, row, lane, j, y[j], r[j], gate[j]);
        if (c.gate) {
            gate[j].get(8 * (lane + TPR * j), K, f);
#pragma unroll
            for (int e = 0; e < 8; ++e) v[j][e] *= f[e];
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) f[e] = 0.0f;
        if (c.r) r[j].get(8 * (lane + TPR * j), K, f);
#pragma unroll
        for (int e = 0; e < 8; e += 2) {
            v[j][e] = fmaf(c.scale, v[j][e], f[e]);
            v[j][e + 1] = fmaf(c.scale, v[j][e + 1], f[e + 1]);
            s0 = fmaf(v[j][e], v[j][e], s0);
            s1 = fmaf(v[j][e + 1], v[j][e + 1], s1);
        }
    }
    if (c.r_out) store_row<XT, VEC, TPR, NV>(static_cast<uint8_t*>(c.r_out) + row * c.ldro * x_size(XT), lane, K, v);
    // past the row's end (k >= K) y, r and gate are 0, so the values are; a weight offset does not reach them
    weigh<VEC, TPR, NV>(c, c.pre, root_of(sum_row<TPR>(s0 + s1, red[1]), c), lane, v);
    if (!c.codes) {
        store_row<XT, VEC, TPR, NV>(static_cast<uint8_t*>(c.h) + row * c.ldh * x_size(XT), lane, K, v);
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
    const bool whole = (reinterpret_cast<uintptr_t>(to) & 7) == 0;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
        const int k = 8 * (lane + TPR * j);
        const uint2 u = qc_codes8(v[j], id);
        if ((VEC || whole) && k + 8 <= K) {
            *reinterpret_cast<uint2*>(to + k) = u;
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e)
                if (k + e < K) to[k + e] = (int8_t)((e < 4 ? u.x : u.y) >> (8 * (e & 3)));
        }
    }
    if (lane == 0) c.scales[row] = d;
}

// ------------------------------------------------------------------ many rows

using Pair = unsigned long long;  // two floats, one instruction for both

// Eight values as they come from memory.
template <int XT>
struct Raw8 {
    uint4 u[XT == X_F32 ? 2 : 1];
    __device__ __forceinline__ void load(const void* row, int k) {
        const uint4* p = reinterpret_cast<const uint4*>(static_cast<const uint8_t*>(row) + (long long)k * x_size(XT));
        u[0] = p[0];
        if constexpr (XT == X_F32) u[1] = p[1];
    }
    __device__ __forceinline__ void zero() {
        u[0] = make_uint4(0u, 0u, 0u, 0u);
        if constexpr (XT == X_F32) u[1] = u[0];
    }
    __device__ __forceinline__ void get(Pair f[4]) const {
        if constexpr (XT == X_F32) {
            f[0] = f2pack(__uint_as_float(u[0].x), __uint_as_float(u[0].y)), f[1] = f2pack(__uint_as_float(u[0].z), __uint_as_float(u[0].w));
            f[2] = f2pack(__uint_as_float(u[1].x), __uint_as_float(u[1].y)), f[3] = f2pack(__uint_as_float(u[1].z), __uint_as_float(u[1].w));
        } else {
            const uint32_t w[4] = {u[0].x, u[0].y, u[0].z, u[0].w};
            float v[8];
            qc_words8<XT>(w, v);
#pragma unroll
            for (int i = 0; i < 4; ++i) f[i] = f2pack(v[2 * i], v[2 * i + 1]);
        }
    }
};
__device__ __forceinline__ void unpack8(const Pair p[4], float f[8]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        f[2 * i] = f2lo(p[i]);
        f[2 * i + 1] = f2hi(p[i]);
    }
}

// What rows share: weights, and a gate per channel.
template <int XT, int WT, int NV>
struct NormWeights {
    Raw8<WT> post[NV], pre[NV];
    Raw8<XT> gate[NV];
};

// Two sums over a row's threads at one barrier.
template <int TPR>
__device__ __forceinline__ void sum_rows(float& a, float& b, float (*red)[32]) {
#pragma unroll
    for (int o = 16; o; o >>= 1) {
        a += __shfl_xor_sync(0xffffffffu, a, o);
        b += __shfl_xor_sync(0xffffffffu, b, o);
    }
    if constexpr (TPR > 32) {
        if ((threadIdx.x & 31) == 0) {
            red[0][threadIdx.x >> 5] = a;
            red[1][threadIdx.x >> 5] = b;
        }
        __syncthreads();
        a = red[0][threadIdx.x & (TPR / 32 - 1)];
        b = red[1][threadIdx.x & (TPR / 32 - 1)];
#pragma unroll
        for (int o = TPR / 64; o; o >>= 1) {
            a += __shfl_xor_sync(0xffffffffu, a, o);
            b += __shfl_xor_sync(0xffffffffu, b, o);
        }
    }
}

template <int XT, int NV>
__device__ __forceinline__ float squares(const Raw8<XT> y[NV]) {
    Pair ss = 0;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
        Pair f[4];
        y[j].get(f);
#pragma unroll
        for (int e = 0; e < 4; ++e) ss = fma2(f[e], f[e], ss);
    }
    return f2lo(ss) + f2hi(ss);
}

// One row, from its values to the outputs.  root: 1 / sqrt(mean(y^2) + eps) of this row; AHEAD: becomes that of
// the next one, whose y next() gives (before the barrier): the sums of r'^2 and of the next y^2 are one
// exchange.  red: three areas of TPR / 32 words, for this row alone until the next but one.  read():
// called when every thread has its values.
template <int XT, int WT, int TPR, int NV, bool POST, bool GATE, bool AHEAD, class Next, class Read>
__device__ __forceinline__ void norm_row(const NormCall& c, long long row, int lane, Raw8<XT> y[NV], const Raw8<XT> r[NV], const Raw8<XT> gate[NV],
                                         const NormWeights<XT, WT, NV>& w, float& root, float (*red)[32], Next next, Read read) {
    const Pair offset = f2pack(c.offset, c.offset), scale = f2pack(c.scale, c.scale), rs = f2pack(root, root);
    Pair v[NV][4], ss = 0;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
        y[j].get(v[j]);
        Pair f[4];
        if (POST) {
            w.post[j].get(f);
#pragma unroll
            for (int e = 0; e < 4; ++e) v[j][e] = mul2(mul2(v[j][e], rs), add2(offset, f[e]));
        }
        if (GATE) {
            gate[j].get(f);
#pragma unroll
            for (int e = 0; e < 4; ++e) v[j][e] = mul2(v[j][e], f[e]);
        }
        r[j].get(f);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            v[j][e] = fma2(scale, v[j][e], f[e]);
            ss = fma2(v[j][e], v[j][e], ss);
        }
    }
    if (c.r_out) {
        uint8_t* to = static_cast<uint8_t*>(c.r_out) + row * c.ldro * x_size(XT);
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            float f[8];
            unpack8(v[j], f);
            if (8 * (lane + TPR * j) < c.K) store8<XT>(to, 8 * (lane + TPR * j), c.K, f);
        }
    }
    next(y);
    float mine = f2lo(ss) + f2hi(ss), other = POST && AHEAD ? squares<XT, NV>(y) : 0.0f;
    if (POST && AHEAD) sum_rows<TPR>(mine, other, red);
    else mine = sum_row<TPR>(mine, TPR > 32 ? red[0] : nullptr);
    read();
    const float own = root_of(mine, c);
    const Pair rs2 = f2pack(own, own);
    if (POST && AHEAD) root = root_of(other, c);
    uint8_t* to = static_cast<uint8_t*>(c.h) + row * c.ldh * x_size(XT);
    uint32_t top = 0;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
        Pair f[4];
        w.pre[j].get(f);
#pragma unroll
        for (int e = 0; e < 4; ++e) v[j][e] = mul2(mul2(v[j][e], rs2), add2(offset, f[e]));
        const bool on = 8 * (lane + TPR * j) < c.K;
        float h[8];
        unpack8(v[j], h);
        if (!c.codes) {
            if (on) store8<XT>(to, 8 * (lane + TPR * j), c.K, h);
        } else if (on) {
#pragma unroll
            for (int e = 0; e < 8; ++e) top = max(top, qc_abs_bits(h[e]));
        }
    }
    if (!c.codes) return;
    float d, id;
    qc_row_scale(max_row<TPR>(top, TPR > 32 ? reinterpret_cast<uint32_t*>(red[2]) : nullptr), d, id);
    int8_t* codes = c.codes + row * c.ldh;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
        float h[8];
        unpack8(v[j], h);
        if (8 * (lane + TPR * j) < c.K) *reinterpret_cast<uint2*>(codes + 8 * (lane + TPR * j)) = qc_codes8(h, id);
    }
    if (lane == 0) c.scales[row] = d;
}

template <int XT, int WT, int TPR, int NV, bool POST, bool GATE>
__device__ __forceinline__ void norm_weights(const NormCall& c, int lane, NormWeights<XT, WT, NV>& w) {
#pragma unroll
    for (int j = 0; j < NV; ++j) {
        const int k = 8 * (lane + TPR * j);
        w.pre[j].zero();
        w.post[j].zero();
        w.gate[j].zero();
        if (k >= c.K) continue;
        w.pre[j].load(c.pre, k);
        if (POST) w.post[j].load(c.post, k);
        if (GATE && c.ldg == 0) w.gate[j].load(c.gate, k);
    }
}

// Short rows: a warp each.
template <int XT, int WT, int NV, bool POST, bool GATE>
__global__ void __launch_bounds__(256, 2) norm_warps_kernel(const NormCall c) {
    grid_dep_launch();
    const int lane = threadIdx.x & 31;
    float(*red)[32] = nullptr;  // one warp: no exchange in shared memory
    grid_dep_wait();
    NormWeights<XT, WT, NV> w;
    norm_weights<XT, WT, 32, NV, POST, GATE>(c, lane, w);
    const long long step = (long long)gridDim.x * 8;
    long long row = (long long)blockIdx.x * 8 + (threadIdx.x >> 5);
    const bool per_row = GATE && c.ldg != 0;
    Raw8<XT> y[NV], r[NV], gate[NV];
    auto load = [&](long long at) {
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int k = 8 * (lane + 32 * j);
            y[j].zero();
            r[j].zero();
            if (GATE) gate[j] = w.gate[j];
            if (at >= c.T || k >= c.K) continue;
            y[j].load(static_cast<const uint8_t*>(c.y) + at * c.ldy * x_size(XT), k);
            if (c.r) r[j].load(static_cast<const uint8_t*>(c.r) + at * c.ldr * x_size(XT), k);
            if (per_row) gate[j].load(static_cast<const uint8_t*>(c.gate) + at * c.ldg * x_size(XT), k);
        }
    };
    load(row);
    for (; row < c.T; row += step) {
        Raw8<XT> y0[NV], r0[NV], g0[NV];
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            y0[j] = y[j];
            r0[j] = r[j];
            if (GATE) g0[j] = gate[j];
        }
        load(row + step);  // outputs may be inputs of their own row, not of another
        float root = 0.0f;  // the next row's sum would wait for its values
        if (POST) root = root_of(sum_row<32>(squares<XT, NV>(y0), nullptr), c);
        norm_row<XT, WT, 32, NV, POST, GATE, false>(c, row, lane, y0, r0, g0, w, root, red, [](Raw8<XT>*) {}, [] {});
    }
}

// blocks an SM
__host__ __device__ constexpr int norm_blocks(int tpr, int nv) { return tpr == 256 && nv == 2 ? 3 : 1024 / tpr; }

// Long rows: a block each, `depth` of them in its ring.
struct NormRing {
    int depth, stage;     // rows; bytes of one's inputs
    unsigned* err;
};
template <int XT, int WT, int TPR, int NV, bool POST, bool GATE>
__global__ void __launch_bounds__(TPR, norm_blocks(TPR, NV)) norm_ring_kernel(const NormCall c, const NormRing q) {
    extern __shared__ __align__(128) uint8_t ring[];
    __shared__ float red[2][3][32];
    __shared__ uint64_t bars[8];
    __shared__ int abort_flag;
    const int tid = threadIdx.x;
    const uint32_t bytes = (uint32_t)c.K * x_size(XT);
    const bool per_row = GATE && c.ldg != 0;
    if (tid == 0) {
        for (int i = 0; i < q.depth; ++i) mbar_init(smem_u32(&bars[i]), 1);
        abort_flag = 0;
        fence_mbar_init();
    }
    grid_dep_launch();
    __syncthreads();
    grid_dep_wait();
    auto ask = [&](long long row, int s) {  // one thread
        const uint32_t bar = smem_u32(&bars[s]), to = smem_u32(ring + (long long)s * q.stage);
        mbar_arrive_tx(bar, (uint32_t)q.stage);
        bulk_g2s(to, static_cast<const uint8_t*>(c.y) + row * c.ldy * x_size(XT), bytes, bar);
        if (c.r) bulk_g2s(to + bytes, static_cast<const uint8_t*>(c.r) + row * c.ldr * x_size(XT), bytes, bar);
        if (per_row) bulk_g2s(to + (uint32_t)q.stage - bytes, static_cast<const uint8_t*>(c.gate) + row * c.ldg * x_size(XT), bytes, bar);
    };
    if (tid == 0)
        for (int i = 0; i < q.depth; ++i)
            if (blockIdx.x + (long long)i * gridDim.x < c.T) ask(blockIdx.x + (long long)i * gridDim.x, i);
    NormWeights<XT, WT, NV> w;
    norm_weights<XT, WT, TPR, NV, POST, GATE>(c, tid, w);
    int s = 0, flip = 0;  // this row's stage; the areas that its sums use
    uint32_t parity = 0;
    Raw8<XT> y[NV];
    // after a wait that gave up (the error word is raised) the results are undefined, and no later wait lasts
    auto take = [&](Raw8<XT>* to, int stage, uint32_t phase) {
        mbar_wait(smem_u32(&bars[stage]), phase, &abort_flag, q.err);
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            to[j].zero();
            if (8 * (tid + TPR * j) < c.K) to[j].load(ring + (long long)stage * q.stage, 8 * (tid + TPR * j));
        }
    };
    take(y, 0, 0);
    float root = 0.0f;
    if (POST) root = root_of(sum_row<TPR>(squares<XT, NV>(y), red[1][2]), c);
    for (long long row = blockIdx.x; row < c.T; row += gridDim.x, flip ^= 1) {
        const uint8_t* from = ring + (long long)s * q.stage;
        Raw8<XT> r[NV], gate[NV];
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int k = 8 * (tid + TPR * j);
            r[j].zero();
            if (GATE) gate[j] = w.gate[j];
            if (k >= c.K) continue;
            if (c.r) r[j].load(from + bytes, k);
            if (per_row) gate[j].load(from + q.stage - bytes, k);
        }
        const int mine = s;
        if (++s == q.depth) {
            s = 0;
            parity ^= 1u;
        }
        norm_row<XT, WT, TPR, NV, POST, GATE, true>(c, row, tid, y, r, gate, w, root, red[flip],
                                              [&](Raw8<XT>* to) {
                                                  if (row + gridDim.x < c.T) take(to, s, parity);
                                              },
                                              [&] {  // this row's stage has been read
                                                  const long long next = row + (long long)q.depth * gridDim.x;
                                                  if (tid == 0 && next < c.T && !abort_flag) ask(next, mine);
                                              });
    }
    if (abort_flag && tid == 0)  // what was asked for lands before the block's memory is given back
        for (int i = 0; i < q.depth; ++i) mbar_drain(smem_u32(&bars[i]), i < s ? parity ^ 1u : parity, &abort_flag, q.err);
}

template <int XT, int WT, int TPR, int NV, bool POST, bool GATE>
cudaError_t ring_one(const NormCall& c, int sms, int smem_max, unsigned* err, cudaStream_t s) {
    static unsigned long long done = 0;
    auto* k = norm_ring_kernel<XT, WT, TPR, NV, POST, GATE>;
    const cudaError_t e = ensure_smem(k, smem_max - 1024, done);
    if (e != cudaSuccess) return e;
    NormRing q;
    q.stage = c.K * x_size(XT) * (1 + (c.r != nullptr) + (GATE && c.ldg != 0));
    q.err = err;
    int per = norm_blocks(TPR, NV);  // blocks an SM: as many as registers allow, three rows each if shared memory does
    while (per > 1 && (smem_max / per - 2048) / q.stage < 3) --per;
    q.depth = (smem_max / per - 2048) / q.stage;
    if (q.depth > 8) q.depth = 8;
    const long long most = (long long)sms * per;
    return launch_pdl(k, (unsigned)(c.T < most ? c.T : most), TPR, (size_t)q.depth * q.stage, s, c, q);
}
template <int XT, int WT, int NV, bool POST, bool GATE>
cudaError_t warps_one(const NormCall& c, int sms, cudaStream_t s) {
    const long long most = 3ll * sms, rows = (c.T + 7ll) / 8;
    return launch_pdl(norm_warps_kernel<XT, WT, NV, POST, GATE>, (unsigned)(rows < most ? rows : most), 256, 0, s, c);
}

// A warp a row while its values fit the registers, which is up to 768 of 16 bits and 256 of f32 (rows of 576: 4323
// in f16 8.2 us, with a ring of 128 threads 9.7; in f32 24 and 13); then blocks of as many threads as a row has
// pieces, but for 16-bit rows of 4096 two pieces each (4096 rows 25.1 us, with 512 threads 27.6; in f32 53.6 and 49.4).
template <int XT, int WT, bool POST, bool GATE>
cudaError_t many_go(const NormCall& c, int sms, int smem_max, unsigned* err, cudaStream_t s) {
    if (c.K <= 256) return warps_one<XT, WT, 1, POST, GATE>(c, sms, s);
    if constexpr (XT != X_F32) {
        if (c.K <= 512) return warps_one<XT, WT, 2, POST, GATE>(c, sms, s);
        if (c.K <= 768) return warps_one<XT, WT, 3, POST, GATE>(c, sms, s);
    }
    if (c.K <= 1024) return ring_one<XT, WT, 128, 1, POST, GATE>(c, sms, smem_max, err, s);
    if (c.K <= 2048) return ring_one<XT, WT, 256, 1, POST, GATE>(c, sms, smem_max, err, s);
    if (c.K <= 4096) {
        if constexpr (XT == X_F32) return ring_one<XT, WT, 512, 1, POST, GATE>(c, sms, smem_max, err, s);
        else return ring_one<XT, WT, 256, 2, POST, GATE>(c, sms, smem_max, err, s);
    }
    return ring_one<XT, WT, 1024, 1, POST, GATE>(c, sms, smem_max, err, s);
}
template <int XT, int WT>
cudaError_t many(const NormCall& c, int sms, int smem_max, unsigned* err, cudaStream_t s) {
    if (c.post) return c.gate ? many_go<XT, WT, true, true>(c, sms, smem_max, err, s) : many_go<XT, WT, true, false>(c, sms, smem_max, err, s);
    return c.gate ? many_go<XT, WT, false, true>(c, sms, smem_max, err, s) : many_go<XT, WT, false, false>(c, sms, smem_max, err, s);
}
template <int XT, int TPR, int NV, bool VEC>
cudaError_t few_one(const NormParams& p, cudaStream_t s) {
    constexpr int rows = TPR == 32 ? 2 : 1;
    return launch_pdl(block_norm_kernel<XT, TPR, NV, VEC>, (unsigned)((p.c.T + (long long)rows - 1) / rows), TPR * rows, 0, s, p);
}
template <int XT, bool VEC>
cudaError_t few(const NormParams& p, cudaStream_t s) {  // threads and pieces: many_go's
    const int K = p.c.K;
    if (K <= 256) return few_one<XT, 32, 1, VEC>(p, s);
    if constexpr (XT != X_F32) {
        if (K <= 512) return few_one<XT, 32, 2, VEC>(p, s);
        if (K <= 768) return few_one<XT, 32, 3, VEC>(p, s);
    }
    if (K <= 1024) return few_one<XT, 128, 1, VEC>(p, s);
    if (K <= 2048) return few_one<XT, 256, 1, VEC>(p, s);
    if (K <= 4096) {
        if constexpr (XT == X_F32) return few_one<XT, 512, 1, VEC>(p, s);
        else return few_one<XT, 256, 2, VEC>(p, s);
    }
    if (K <= 8192) return few_one<XT, 1024, 1, VEC>(p, s);
    if (K <= 16384) return few_one<XT, 1024, 2, VEC>(p, s);  // 16 x 14336 bf16 5.0 us, with four pieces 8.2
    return few_one<XT, 1024, 4, VEC>(p, s);
}

// Rows of up to 4096 (f32: 256) go to the kernels for many rows however few they are, longer ones from two an SM on
// (block_norm_kernel / those, us, norm on both sides): bf16 1 x 576 3.8 / 2.1, 611 x 576 4.3 / 2.7, 16 x 4096 3.3 / 2.6,
// 304 x 4096 5.5 / 4.8, 152 x 8192 4.9 / 5.1, 304 x 8192 9.2 / 7.4; f32 1216 x 256 2.6 / 2.2, 16 x 2048 2.4 / 2.6,
// 304 x 2048 5.1 / 4.4, 4323 x 576 18 / 13, 64 x 8192 5.0 / 6.0.
template <int XT>
cudaError_t norm_go(const NormParams& p, cudaStream_t s) {
    const int K = p.c.K;
    int sms = 0, smem = 0;
    unsigned* err = nullptr;
    const cudaError_t e = device_constants(&err, &sms, &smem);
    if (e != cudaSuccess) return e;
    if (p.vec && K % 8 == 0 && K <= 8192 && (K <= (XT == X_F32 ? 256 : 4096) || p.c.T >= 2 * sms)) {
        if (p.c.wt == XT) return many<XT, XT>(p.c, sms, smem, err, s);
        if (p.c.wt == X_F32) return many<XT, X_F32>(p.c, sms, smem, err, s);
    }
    return p.vec ? few<XT, true>(p, s) : few<XT, false>(p, s);
}

}  // namespace
}  // namespace qmm
