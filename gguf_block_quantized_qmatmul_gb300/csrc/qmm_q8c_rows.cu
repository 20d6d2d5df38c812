// qmm_q8c_rows.cu -- 8-bit channel-scaled products of up to four activation
// rows.
//
// Mathematics.  Integer warp MMAs (16 weight rows x 32 K x 8 columns, int32
// sums: exact for every K that the layout takes) on the codes as they are; a
// row block's int32 sums are added where warps split it, and one f32 expression
// makes a result of it (qc_scale).
//
// Bound by the weight stream, a byte a weight.  One persistent block an SM
// over an equal share of the row blocks, whose segments are dealt to its warps in
// equal contiguous runs, wherever row blocks end; every warp streams its own
// through a ring of asynchronous 16-byte copies, two conflict-free 16-byte loads
// a lane and tile, no conversion, and waits for no other until the parts of cut
// row blocks are added at the end.  The integer MMAs (152 TOPS on this GPU) would
// take 25 us of the 35 that the weights of 28672 x 8192 take from memory.
// Activations are staged once, as codes, 64 bytes a tile and row (rows a
// multiple of 128 plus 64 bytes apart: no bank conflicts).  Up to 16384 values
// are quantized by every block for itself, as a second launch costs more (one row of
// 4096 x 4096: 7.6 us, with it 10.4).  Few of them leave a block of 8 warps the
// faster one: two such blocks fit an SM, so that the next call's first weights
// are on their way before this one ends (7.6 us; with 16 warps 9.3); 16 warps
// stage more values sooner (4 rows of 14336 x 4096: 15.8 us, with 8 18.5).
// Weights are constant, so their first copies are issued before the grid that
// this one depends on has completed.
//
// Measured: one row of 28672 x 8192 bf16 41 us (5.7 TB/s), of 14336 x 4096 13.8.
#include "qmm_q8c.cuh"
#include "qmm_q4g_rows.cuh"

namespace qmm {
namespace {

constexpr int kDepth = 4;       // segments in a warp's ring
constexpr int kMaxWarps = 16;
constexpr int kMaxRows = 4;
constexpr int kStatic = 1024;   // the kernel's static arrays, rounded up

struct RowsParams {
    QcCall c;
    int pitch, quant, warps_log2;
    int kx;  // columns of codes that are there to be read: K, or the padded row of the preparation
    int off_zero, off_part, off_ring;
};

__device__ __forceinline__ void mma_s8_add(int d[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k32.row.col.s32.s8.s8.s32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+r"(d[0]), "+r"(d[1]), "+r"(d[2]), "+r"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Eight values as they come from memory: two 16-byte words of f32, one of 16-bit floats.
template <int XT>
__device__ __forceinline__ void raw_floats(const uint4 u[2], float f[8]) {
    if constexpr (XT == X_F32) {
        f[0] = __uint_as_float(u[0].x), f[1] = __uint_as_float(u[0].y), f[2] = __uint_as_float(u[0].z), f[3] = __uint_as_float(u[0].w);
        f[4] = __uint_as_float(u[1].x), f[5] = __uint_as_float(u[1].y), f[6] = __uint_as_float(u[1].z), f[7] = __uint_as_float(u[1].w);
    } else {
        const uint32_t w[4] = {u[0].x, u[0].y, u[0].z, u[0].w};
        qc_words8<XT>(w, f);
    }
}

// Quantizes the rows into shared memory; top: a word per row.  Rows are aligned, K a multiple of 8.  Two
// trips over the values (one, where they fit the registers), four pieces of 8 a thread in flight.
template <int XT>
__device__ __forceinline__ void stage_floats(uint8_t* sm, float* scale, uint32_t* top, const RowsParams& p, int tid, int nthr) {
    const int rows = p.c.a.M, n8 = p.c.w.KS * 16, n = rows * n8, K = p.c.w.K;  // pieces of 8 values; a half warp's are one row's
    const uint8_t* x = static_cast<const uint8_t*>(p.c.a.x);
    if (tid < rows) top[tid] = 0u;
    __syncthreads();
    uint4 u[4][2];
    const bool once = n <= 4 * nthr;  // the values stay in registers
#pragma unroll 1
    for (int pass = 0; pass < 2; ++pass) {
#pragma unroll 1
        for (int i0 = 0; i0 < n; i0 += 4 * nthr) {
            if (pass == 0 || !once) {
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const int i = i0 + j * nthr + tid, r = i / n8, k = 8 * (i - r * n8);
                    u[j][0] = u[j][1] = make_uint4(0u, 0u, 0u, 0u);
                    if (i >= n || k >= K) continue;
                    const uint4* from = reinterpret_cast<const uint4*>(x + (r * p.c.a.ld + k) * x_size(XT));
                    u[j][0] = *from;
                    if (XT == X_F32) u[j][1] = from[1];
                }
            }
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int i = i0 + j * nthr + tid, r = i / n8;
                if (i - (tid & 31) >= n) break;  // the whole warp is done
                float f[8];
                raw_floats<XT>(u[j], f);
                if (pass == 0) {
                    uint32_t m = 0;
#pragma unroll
                    for (int e = 0; e < 8; ++e) m = max(m, qc_abs_bits(f[e]));
#pragma unroll
                    for (int o = 8; o; o >>= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, o));
                    if ((tid & 15) == 0 && i < n) atomicMax(&top[r], m);
                } else if (i < n) {
                    float d, id;
                    qc_row_scale(top[r], d, id);
                    *reinterpret_cast<uint2*>(sm + r * p.pitch + 8 * (i - r * n8)) = qc_codes8(f, id);
                    if (i == r * n8) scale[r] = d;
                }
            }
        }
        __syncthreads();
    }
}

// Codes that are there: rows on 16-byte boundaries, K a multiple of 16.
__device__ __forceinline__ void stage_codes(uint8_t* sm, float* scale, const RowsParams& p, int tid, int nthr) {
    const QcRows& a = p.c.a;
    const int n16 = p.c.w.KS * 8, n = a.M * n16;
    const uint8_t* x = static_cast<const uint8_t*>(a.x);
    for (int i0 = 0; i0 < n; i0 += 4 * nthr) {
        uint4 v[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int i = i0 + j * nthr + tid, r = i / n16, k = 16 * (i - r * n16);
            v[j] = make_uint4(0u, 0u, 0u, 0u);
            if (i < n && k < p.kx) v[j] = *reinterpret_cast<const uint4*>(x + r * a.ld + k);
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int i = i0 + j * nthr + tid, r = i / n16, k = 16 * (i - r * n16);
            if (i < n) *reinterpret_cast<uint4*>(sm + r * p.pitch + k) = v[j];
        }
    }
    if (tid < a.M) scale[tid] = a.scales[tid];
}

__global__ void __launch_bounds__(kMaxWarps * 32, 1) q8c_rows_kernel(const RowsParams p) {
    extern __shared__ __align__(16) uint8_t sm[];
    __shared__ uint32_t top[kMaxRows];
    __shared__ float scale[kMaxRows];
    const QcCall& c = p.c;
    const QcWeights& w = c.w;
    const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31, g = lane >> 2, t = lane & 3, nthr = blockDim.x;
    const int KS = w.KS, M = c.a.M;
    uint8_t* ring = sm + p.off_ring + warp * (kDepth * kQcSeg);
    int4* parts = reinterpret_cast<int4*>(sm + p.off_part);  // [warp][2][32]: a row block's part that does not reach its end: 1; that does: 0
    if (tid == 0) *reinterpret_cast<uint4*>(sm + p.off_zero) = make_uint4(0u, 0u, 0u, 0u);  // what lanes without a column read
    grid_dep_launch();

    // an equal share of the row blocks a block, and of its segments a warp
    const int rb0 = (int)(blockIdx.x * (unsigned)w.RB / gridDim.x), rb1 = (int)((blockIdx.x + 1) * (unsigned)w.RB / gridDim.x);  // RB <= 2^19
    const float* sw = reinterpret_cast<const float*>(w.data + w.scale_off);
    const int total = (rb1 - rb0) * KS;
    auto begin = [&](int o) { return (int)((long long)o * total >> p.warps_log2); };  // of warp o's segments
    const int s0 = begin(warp), s1 = begin(warp + 1);
    int left = s1 - s0, ls = 0, lrb = rb0 + s0 / KS, lrem = KS - s0 % KS, step = qc_step(w, lrb);
    const uint8_t* lp = w.data + qc_row_block(w, lrb) + (long long)(KS - lrem) * step + lane * 16;
    const uint32_t to = smem_u32(ring) + lane * 16;
    auto load = [&]() {  // a group of copies, empty past the end, so that the groups' count is the ring's
        if (left > 0) {
            --left;
            const uint32_t d = to + ls * kQcSeg;
#pragma unroll
            for (int i = 0; i < 4; ++i) cp_async16(d + 512 * i, lp + 512 * i);
            lp += step;
            if (--lrem == 0) {  // the next row block
                lrem = KS;
                step = qc_step(w, ++lrb);
                lp = w.data + qc_row_block(w, lrb) + lane * 16;
            }
        }
        ls = ls + 1 == kDepth ? 0 : ls + 1;
        cp_async_commit();
    };
#pragma unroll
    for (int i = 0; i < kDepth - 1; ++i) load();
    grid_dep_wait();
    if (!p.quant) stage_codes(sm, scale, p, tid, nthr);
    else if (c.a.xt == X_F32) stage_floats<X_F32>(sm, scale, top, p, tid, nthr);
    else if (c.a.xt == X_F16) stage_floats<X_F16>(sm, scale, top, p, tid, nthr);
    else stage_floats<X_BF16>(sm, scale, top, p, tid, nthr);
    __syncthreads();

    // what a row block's results need besides their sums, asked for when the row block begins
    float w0 = 0.0f, w1 = 0.0f, b0 = 0.0f, b1 = 0.0f;
    auto ask = [&](int rb) {
        const int n = rb * 16 + g;
        const bool on0 = n < w.N, on1 = n + 8 < w.N;
        w0 = on0 ? __ldg(sw + n) : 0.0f;
        w1 = on1 ? __ldg(sw + n + 8) : 0.0f;
        b0 = c.bias && on0 ? c.bias[n] : 0.0f;
        b1 = c.bias && on1 ? c.bias[n + 8] : 0.0f;
    };
    // a row block's 16 x 8 sums to their places: column 2 t + i, rows g and g + 8
    auto put = [&](const int v[4], int rb) {
        const int n = rb * 16 + g;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int r = 2 * t + i;
            if (r >= M) continue;
            const float sx = scale[r];
            const long long o = (long long)r * w.N + n;
            if (n < w.N) x_store(c.y, c.yt, o, qc_scale((float)v[i], w0, sx, b0));
            if (n + 8 < w.N) x_store(c.y, c.yt, o + 8, qc_scale((float)v[2 + i], w1, sx, b1));
        }
    };
    int acc[4] = {0, 0, 0, 0};
    int cut = -1, cut_rb = 0;  // the row block that this warp completes but did not begin: its first one
    float cut_w0 = 0.0f, cut_w1 = 0.0f, cut_b0 = 0.0f, cut_b1 = 0.0f;
    int cs = 0, seg = s0 % KS, rb = rb0 + s0 / KS;  // ring place; segment in the row block
    bool began = seg == 0;
    // this lane's column g, xq bytes from a tile to the next (0: it has no column)
    const int xq = g < M ? 64 : 0, xp = g < M ? g * p.pitch + t * 16 : p.off_zero;
    for (int i = s0; i < s1; seg = 0, ++rb) {
        const int from = i - seg, end = min(s1, from + KS);
        const bool done = end == from + KS;
        if (done) ask(rb);
        const uint8_t* xs = sm + xp + 2 * seg * xq;
        for (; i < end; ++i) {
            cp_async_wait<kDepth - 2>();
            __syncwarp();  // every lane's copies of this segment have landed, and the last one has been read
            load();
            const uint8_t* sp = ring + cs * kQcSeg + lane * 16;
            cs = cs + 1 == kDepth ? 0 : cs + 1;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const uint4 a = *reinterpret_cast<const uint4*>(sp + 1024 * h), e = *reinterpret_cast<const uint4*>(sp + 1024 * h + 512);
                const uint4 xv = *reinterpret_cast<const uint4*>(xs + h * xq);
                mma_s8_add(acc, a.x, e.x, a.y, e.y, xv.x, xv.y);
                mma_s8_add(acc, a.z, e.z, a.w, e.w, xv.z, xv.w);
            }
            xs += 2 * xq;
        }
        if (done && began) {
            put(acc, rb);
        } else {
            parts[(warp * 2 + (done ? 0 : 1)) * 32 + lane] = make_int4(acc[0], acc[1], acc[2], acc[3]);
            if (done) {
                cut = from;
                cut_rb = rb;
                cut_w0 = w0, cut_w1 = w1, cut_b0 = b0, cut_b1 = b1;
            }
        }
        began = true;
        acc[0] = acc[1] = acc[2] = acc[3] = 0;
    }
    cp_async_wait<0>();
    __syncthreads();  // all parts are there
    if (cut >= 0) {
        int o = warp - 1;
        while (begin(o) > cut) --o;
        for (; o <= warp; ++o) {
            if (begin(o) == begin(o + 1)) continue;  // no segments
            const int4 u = parts[(o * 2 + (o == warp ? 0 : 1)) * 32 + lane];
            acc[0] += u.x;
            acc[1] += u.y;
            acc[2] += u.z;
            acc[3] += u.w;
        }
        w0 = cut_w0, w1 = cut_w1, b0 = cut_b0, b1 = cut_b1;
        put(acc, cut_rb);
    }
}

// Whether the blocks stage these activations themselves.
bool rows_direct(const QcRows& a, int K) {
    const long long size = a.scales ? 1 : x_size(a.xt);
    if ((reinterpret_cast<uintptr_t>(a.x) | (uintptr_t)(a.ld * size)) % 16 != 0 || K % (a.scales ? 16 : 8) != 0) return false;
    return a.scales || (long long)a.M * K <= 16384;
}

}  // namespace

QcRowsPlan plan_q8c_rows(const QcCall& c, int sms, int smem_max) {
    QcRowsPlan pl;
    const QcWeights& w = c.w;
    if (c.a.M > kMaxRows || (long long)w.RB * w.KS > INT32_MAX) return pl;
    pl.pitch = w.KS * 128 + 64;
    const int act = c.a.M * pl.pitch, room = smem_max - kStatic - 1024 - 16 - act, per_warp = 1024 + kDepth * kQcSeg;
    pl.warps = (long long)c.a.M * w.K <= 8192 || kMaxWarps * per_warp > room ? 8 : kMaxWarps;  // beside long rows eight fit
    const int rest = pl.warps * per_warp;
    if (rest > room) return pl;
    pl.blocks = w.RB < sms ? w.RB : sms;
    pl.off_zero = act;
    pl.off_part = pl.off_zero + 16;
    pl.off_ring = pl.off_part + pl.warps * 1024;
    pl.smem = (size_t)act + 16 + rest;
    // what is not read 16 bytes at a time goes through the preparation, as does what would take each
    // block longer than a launch
    pl.prep = !rows_direct(c.a, w.K);
    pl.workspace = pl.prep ? (size_t)c.a.M * w.KS * 128 + 16 : 0;
    pl.ok = true;
    return pl;
}

cudaError_t launch_q8c_rows(const QcRowsPlan& pl, const QcCall& c, void* ws, int smem_max, cudaStream_t s) {
    RowsParams p;
    p.c = c;
    if (pl.prep) {
        uint8_t* codes = static_cast<uint8_t*>(ws);
        const long long pitch = (long long)c.w.KS * 128;
        float* scales = reinterpret_cast<float*>(codes + c.a.M * pitch);
        const cudaError_t e = launch_q8c_prep(c.a, c.w.K, QcPrep{codes, scales, nullptr, pitch}, false, s);
        if (e != cudaSuccess) return e;
        p.c.a = QcRows{codes, scales, pitch, 0, c.a.M};
    }
    p.kx = pl.prep ? c.w.KS * 128 : c.w.K;
    p.quant = p.c.a.scales == nullptr;
    p.pitch = pl.pitch;
    p.warps_log2 = pl.warps == 8 ? 3 : 4;
    p.off_zero = pl.off_zero;
    p.off_part = pl.off_part;
    p.off_ring = pl.off_ring;
    static unsigned long long done = 0;
    const cudaError_t e = ensure_smem(q8c_rows_kernel, smem_max - kStatic, done);
    if (e != cudaSuccess) return e;
    return launch_pdl(q8c_rows_kernel, (unsigned)pl.blocks, (unsigned)(pl.warps * 32), pl.smem, s, p);
}

}  // namespace qmm
