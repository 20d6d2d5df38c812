// qmm_q8c_rows.cu -- 8-bit channel-scaled products of few activation rows.
//
// Mathematics.  Integer warp MMAs (16 weight rows x 32 K x 8 activation rows,
// int32 sums: exact for every K that the layout takes) on the codes as they
// are; a row block's int32 sums are added where warps split it, and one f32
// expression makes a result of it (qc_scale).
//
// Bound by the weight stream, a byte a weight.  One persistent block an SM
// over an equal share of the row blocks, whose segments are dealt to its warps in
// equal contiguous runs, wherever row blocks end; every warp streams its own
// through a ring of asynchronous 16-byte copies, two conflict-free 16-byte loads
// a lane and tile, no conversion, and waits for no other until the parts of cut
// row blocks are added at the end.  The integer MMAs (152 TOPS on
// this GPU) would take 25 us of the 35 that the weights of 28672 x 8192 take
// from memory, for up to 8 rows.
// Activations are staged once, as codes, 64 bytes a tile and row (rows a
// multiple of 128 plus 64 bytes apart: no bank conflicts).  Few values are
// quantized by every block for itself, as a second launch would cost more.
// Weights are constant, so their first copies are issued before the grid that
// this one depends on has completed.
#include <cmath>

#include "qmm_q8c.cuh"
#include "qmm_q4g_rows.cuh"

namespace qmm {
namespace {

constexpr int kDepth = 4;       // segments in a warp's ring
constexpr int kMaxWarps = 16;
constexpr int kStatic = 1024;   // the kernel's static arrays, rounded up

struct RowsParams {
    QcCall c;
    int cols, pitch, quant;
    int kx;  // columns of codes that are there to be read: K, or the padded row of the preparation
    int off_zero, off_scale, off_part, off_ring;
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

// Quantizes `rows` rows (from row m0) into shared memory; top: a word per row.  Rows are aligned, K a
// multiple of 8.  Two trips over the values (one, where they fit the registers), four pieces of 8 a thread in flight.
template <int XT>
__device__ __forceinline__ void stage_floats(uint8_t* sm, float* scale, uint32_t* top, const RowsParams& p, int m0, int rows, int tid, int nthr) {
    const int n8 = p.c.w.KS * 16, n = rows * n8, K = p.c.w.K;  // pieces of 8 values; a half warp's are one row's
    const uint8_t* x = static_cast<const uint8_t*>(p.c.a.x) + m0 * p.c.a.ld * x_size(XT);
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
                    u[j][0] = __ldg(from);
                    if (XT == X_F32) u[j][1] = __ldg(from + 1);
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
__device__ __forceinline__ void stage_codes(uint8_t* sm, float* scale, const RowsParams& p, int m0, int rows, int tid, int nthr) {
    const QcRows& a = p.c.a;
    const int n16 = p.c.w.KS * 8, n = rows * n16;
    const uint8_t* x = static_cast<const uint8_t*>(a.x) + m0 * a.ld;
    for (int i0 = 0; i0 < n; i0 += 4 * nthr) {
        uint4 v[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int i = i0 + j * nthr + tid, r = i / n16, k = 16 * (i - r * n16);
            v[j] = make_uint4(0u, 0u, 0u, 0u);
            if (i < n && k < p.kx) v[j] = __ldg(reinterpret_cast<const uint4*>(x + r * a.ld + k));
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int i = i0 + j * nthr + tid, r = i / n16, k = 16 * (i - r * n16);
            if (i < n) *reinterpret_cast<uint4*>(sm + r * p.pitch + k) = v[j];
        }
    }
    if (tid < rows) scale[tid] = a.scales[m0 + tid];
}

template <int NB>
__global__ void __launch_bounds__(kMaxWarps * 32, 1) q8c_rows_kernel(const RowsParams p) {
    extern __shared__ __align__(16) uint8_t sm[];
    __shared__ uint32_t top[32];
    const QcCall& c = p.c;
    const QcWeights& w = c.w;
    const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31, g = lane >> 2, t = lane & 3, nthr = blockDim.x, warps = nthr >> 5;
    const int KS = w.KS;
    uint8_t* ring = sm + p.off_ring + warp * (kDepth * kQcSeg);
    float* scale = reinterpret_cast<float*>(sm + p.off_scale);
    int4* parts = reinterpret_cast<int4*>(sm + p.off_part);  // [warp][2][NB][32]: a row block's part that does not reach its end: 1; that does: 0
    if (tid == 0) *reinterpret_cast<uint4*>(sm + p.off_zero) = make_uint4(0u, 0u, 0u, 0u);  // what lanes without a column read
    grid_dep_launch();

    const int items = (c.a.M + p.cols - 1) / p.cols;
    const long long work = (long long)items * w.RB;  // row blocks of items, end to end: an equal share a block
    const long long w0 = (long long)blockIdx.x * work / gridDim.x, w1 = (long long)(blockIdx.x + 1) * work / gridDim.x;
    const float* sw = reinterpret_cast<const float*>(w.data + w.scale_off);
    bool waited = false;

    for (long long at = w0; at < w1;) {
        const int item = (int)(at / w.RB), rb0 = (int)(at - (long long)item * w.RB);
        const int rb1 = (int)min((long long)w.RB, rb0 + (w1 - at));
        at += rb1 - rb0;
        const int m0 = item * p.cols, rows = min(p.cols, c.a.M - m0);
        // this warp's segments of the item's row blocks, end to end
        const int total = (rb1 - rb0) * KS, s0 = (int)((long long)warp * total / warps), s1 = (int)((long long)(warp + 1) * total / warps);
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
        if (!waited) {
            grid_dep_wait();
            waited = true;
        }
        if (!p.quant) stage_codes(sm, scale, p, m0, rows, tid, nthr);
        else if (c.a.xt == X_F32) stage_floats<X_F32>(sm, scale, top, p, m0, rows, tid, nthr);
        else if (c.a.xt == X_F16) stage_floats<X_F16>(sm, scale, top, p, m0, rows, tid, nthr);
        else stage_floats<X_BF16>(sm, scale, top, p, m0, rows, tid, nthr);
        __syncthreads();

        // what a row block's results need besides their sums, asked for when the row block begins
        float w0s = 0.0f, w1s = 0.0f, b0 = 0.0f, b1 = 0.0f;
        auto ask = [&](int rb) {
            const int n = rb * 16 + g;
            const bool on0 = n < w.N, on1 = n + 8 < w.N;
            w0s = on0 ? __ldg(sw + n) : 0.0f;
            w1s = on1 ? __ldg(sw + n + 8) : 0.0f;
            b0 = c.bias && on0 ? __ldg(c.bias + n) : 0.0f;
            b1 = c.bias && on1 ? __ldg(c.bias + n + 8) : 0.0f;
        };
        // a row block's 16 x 8 NB sums to their places: column 8 b + 2 t + i, rows g and g + 8
        auto put = [&](const int (&v)[NB][4], int rb) {
            const int n = rb * 16 + g;
            const bool on0 = n < w.N, on1 = n + 8 < w.N;
#pragma unroll
            for (int b = 0; b < NB; ++b)
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const int r = 8 * b + 2 * t + i;
                    if (r >= rows) continue;
                    const float sx = scale[r];
                    const long long o = (long long)(m0 + r) * w.N + n;
                    if (on0) x_store(c.y, c.yt, o, qc_scale((float)v[b][i], w0s, sx, b0));
                    if (on1) x_store(c.y, c.yt, o + 8, qc_scale((float)v[b][2 + i], w1s, sx, b1));
                }
        };
        int acc[NB][4];
        auto clear = [&]() {
#pragma unroll
            for (int b = 0; b < NB; ++b)
#pragma unroll
                for (int i = 0; i < 4; ++i) acc[b][i] = 0;
        };
        clear();
        int cut = -1, cut_rb = 0;  // the row block that this warp completes but did not begin: its first one
        float cut_w0 = 0.0f, cut_w1 = 0.0f, cut_b0 = 0.0f, cut_b1 = 0.0f;
        int cs = 0, seg = s0 % KS, rb = rb0 + s0 / KS;  // ring place; segment in the row block
        bool began = seg == 0;
        for (int i = s0; i < s1; seg = 0, ++rb) {
            const int end = min(s1, i - seg + KS);
            const bool done = end == i - seg + KS;
            // this lane's columns (8 b + g) at xo, xq bytes from a tile to the next (0: it has no column)
            int xo[NB], xq[NB];
#pragma unroll
            for (int b = 0; b < NB; ++b) {
                const bool on = 8 * b + g < rows;
                xq[b] = on ? 64 : 0;
                xo[b] = on ? (8 * b + g) * p.pitch + t * 16 + seg * 128 : p.off_zero;
            }
            const int from = i - seg;
            if (done) ask(rb);
            for (; i < end; ++i) {
                cp_async_wait<kDepth - 2>();
                __syncwarp();  // every lane's copies of this segment have landed, and the last one has been read
                load();
                const uint8_t* sp = ring + cs * kQcSeg + lane * 16;
                cs = cs + 1 == kDepth ? 0 : cs + 1;
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const uint4 a = *reinterpret_cast<const uint4*>(sp + 1024 * h), e = *reinterpret_cast<const uint4*>(sp + 1024 * h + 512);
#pragma unroll
                    for (int b = 0; b < NB; ++b) {
                        const uint4 xv = *reinterpret_cast<const uint4*>(sm + xo[b] + h * xq[b]);
                        mma_s8_add(acc[b], a.x, e.x, a.y, e.y, xv.x, xv.y);
                        mma_s8_add(acc[b], a.z, e.z, a.w, e.w, xv.z, xv.w);
                    }
                }
#pragma unroll
                for (int b = 0; b < NB; ++b) xo[b] += 2 * xq[b];
            }
            if (done && began) {
                put(acc, rb);
            } else {
#pragma unroll
                for (int b = 0; b < NB; ++b) parts[((warp * 2 + (done ? 0 : 1)) * NB + b) * 32 + lane] = make_int4(acc[b][0], acc[b][1], acc[b][2], acc[b][3]);
                if (done) {
                    cut = from;
                    cut_rb = rb;
                    cut_w0 = w0s, cut_w1 = w1s, cut_b0 = b0, cut_b1 = b1;
                }
            }
            began = true;
            clear();
        }
        cp_async_wait<0>();
        __syncthreads();  // all parts are there, and the activations are no longer read
        if (cut >= 0) {
            int o = warp - 1;
            while ((int)((long long)o * total / warps) > cut) --o;
            for (; o <= warp; ++o) {
                if ((int)((long long)o * total / warps) == (int)((long long)(o + 1) * total / warps)) continue;  // no segments
#pragma unroll
                for (int b = 0; b < NB; ++b) {
                    const int4 u = parts[((o * 2 + (o == warp ? 0 : 1)) * NB + b) * 32 + lane];
                    acc[b][0] += u.x;
                    acc[b][1] += u.y;
                    acc[b][2] += u.z;
                    acc[b][3] += u.w;
                }
            }
            w0s = cut_w0, w1s = cut_w1, b0 = cut_b0, b1 = cut_b1;
            put(acc, cut_rb);
        }
        if (at < w1) __syncthreads();  // the parts and the scales have been read
    }
    if (!waited) grid_dep_wait();
}

template <int NB>
cudaError_t rows_go(const QcRowsPlan& pl, const RowsParams& p, int smem_max, cudaStream_t s) {
    static unsigned long long done = 0;
    auto* k = q8c_rows_kernel<NB>;
    const cudaError_t e = ensure_smem(k, smem_max - kStatic, done);
    if (e != cudaSuccess) return e;
    return launch_pdl(k, (unsigned)pl.blocks, (unsigned)(pl.warps * 32), pl.smem, s, p);
}

// Whether the blocks stage these activations themselves.
bool rows_direct(const QcRows& a, int K) {
    const long long size = a.scales ? 1 : x_size(a.xt);
    if ((reinterpret_cast<uintptr_t>(a.x) | (uintptr_t)(a.ld * size)) % 16 != 0 || K % (a.scales ? 16 : 8) != 0) return false;
    return a.scales || (long long)a.M * K <= 32768;
}

}  // namespace

QcRowsPlan plan_q8c_rows(const QcCall& c, int sms, int smem_max) {
    QcRowsPlan pl;
    const QcWeights& w = c.w;
    pl.pitch = w.KS * 128 + 64;
    const long long room = smem_max - kStatic - 1024;
    auto nb_of = [](int cols) { return cols <= 8 ? 1 : cols <= 16 ? 2 : 4; };
    auto fixed = [&](int cols, int warps) { return (long long)round_up(cols * 4, 16) + 16 + warps * 1024ll * nb_of(cols) + (long long)warps * kDepth * kQcSeg; };
    if ((long long)w.RB * w.KS > INT32_MAX) return pl;
    double best = 0;
    for (int most : {8, 16, 32}) {
        int cols = c.a.M < most ? c.a.M : most;
        while (cols > 1 && cols * (long long)pl.pitch + fixed(cols, 8) > room) --cols;
        const int items = (c.a.M + cols - 1) / cols;
        cols = (c.a.M + items - 1) / items;
        const int nb = nb_of(cols);
        for (int warps : {16, 8}) {
            if (cols * (long long)pl.pitch + fixed(cols, warps) > room) continue;
            const long long work = (long long)items * w.RB, blocks = work < sms ? work : sms;
            const double share = (double)((work + blocks - 1) / blocks);  // row blocks
            // segments of a block, more slowly with more columns; a trip to memory and the staging per item
            const double cost = share * w.KS * (nb == 1 ? 1.0 : nb == 2 ? 1.4 : 2.6) * (warps == 8 ? 1.4 : 1.0) + (1.0 + (double)(items - 1) * blocks / (items * (double)blocks)) * (40.0 + cols * w.KS * 0.1);
            if (best == 0 || cost < best) {
                best = cost;
                pl.cols = cols;
                pl.nb = nb;
                pl.warps = warps;
                pl.blocks = (int)blocks;
                pl.items = items;
            }
        }
    }
    if (best == 0) return pl;
    pl.off_zero = pl.cols * pl.pitch;
    pl.off_scale = pl.off_zero + 16;
    pl.off_part = pl.off_scale + round_up(pl.cols * 4, 16);
    pl.off_ring = pl.off_part + pl.warps * 1024 * pl.nb;
    pl.smem = (size_t)pl.off_ring + (size_t)pl.warps * kDepth * kQcSeg;
    // what is not read 16 bytes at a time goes through the preparation, as does what would take each
    // block longer than a launch: see rows_direct
    pl.prep = !rows_direct(c.a, w.K);
    pl.workspace = pl.prep ? (size_t)c.a.M * w.KS * 128 + (size_t)(c.a.M + 3) / 4 * 16 : 0;
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
    p.cols = pl.cols;
    p.pitch = pl.pitch;
    p.off_zero = pl.off_zero;
    p.off_scale = pl.off_scale;
    p.off_part = pl.off_part;
    p.off_ring = pl.off_ring;
    return pl.nb == 1 ? rows_go<1>(pl, p, smem_max, s) : pl.nb == 2 ? rows_go<2>(pl, p, smem_max, s) : rows_go<4>(pl, p, smem_max, s);
}

}  // namespace qmm
