// qmm_q8c_rows.cu -- 8-bit channel-scaled products of few activation rows.
//
// Mathematics.  Integer warp MMAs (16 weight rows x 32 K x 8 activation rows,
// int32 sums: exact for every K that the layout takes) on the codes as they
// are; the warps that split a row block's K add their int32 sums, and one f32
// expression makes a result of it (qc_scale).
//
// Bound by the weight stream, a byte a weight.  One persistent block an SM
// over an equal share of the row blocks; every warp streams its segments
// through its own ring of asynchronous 16-byte copies, two conflict-free
// 16-byte loads a lane and tile, no conversion.  The integer MMAs (152 TOPS on
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
    int cols, wk, wk_log2, wr, pitch, quant;
    int kx;  // columns of codes that are there to be read: K, or the padded row of the preparation
    int off_zero, off_scale, off_red, off_ring;
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
// multiple of 8.  Two trips over the values, four pieces of 8 a thread in flight.
template <int XT>
__device__ __forceinline__ void stage_floats(uint8_t* sm, float* scale, uint32_t* top, const RowsParams& p, int m0, int rows, int tid, int nthr) {
    const int n8 = p.c.w.KS * 16, n = rows * n8, K = p.c.w.K;  // pieces of 8 values; a half warp's are one row's
    const uint8_t* x = static_cast<const uint8_t*>(p.c.a.x) + m0 * p.c.a.ld * x_size(XT);
    if (tid < rows) top[tid] = 0u;
    __syncthreads();
#pragma unroll 1
    for (int pass = 0; pass < 2; ++pass) {
#pragma unroll 1
        for (int i0 = 0; i0 < n; i0 += 4 * nthr) {
            uint4 u[4][2];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int i = i0 + j * nthr + tid, r = i / n8, k = 8 * (i - r * n8);
                u[j][0] = u[j][1] = make_uint4(0u, 0u, 0u, 0u);
                if (i >= n || k >= K) continue;
                const uint4* from = reinterpret_cast<const uint4*>(x + (r * p.c.a.ld + k) * x_size(XT));
                u[j][0] = __ldg(from);
                if (XT == X_F32) u[j][1] = __ldg(from + 1);
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
    const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31, g = lane >> 2, t = lane & 3, nthr = blockDim.x;
    const int wk = p.wk, wr = p.wr, kw = warp & (wk - 1), rw = warp >> p.wk_log2;
    uint8_t* ring = sm + p.off_ring + warp * (kDepth * kQcSeg);
    float* scale = reinterpret_cast<float*>(sm + p.off_scale);
    int* red = reinterpret_cast<int*>(sm + p.off_red);
    constexpr int kRed = NB * 128;  // sums of a warp: [column][16 rows]
    int flip = 0;                   // which of its two areas a row block's sums use
    if (tid == 0) *reinterpret_cast<uint4*>(sm + p.off_zero) = make_uint4(0u, 0u, 0u, 0u);  // what lanes without a column read
    grid_dep_launch();

    const int nit = (w.KS + wk - 1) >> p.wk_log2;  // segments per warp and row block
    const long long rb_bytes = (long long)w.KS * kQcSeg;
    const int items = (c.a.M + p.cols - 1) / p.cols;
    const long long work = (long long)items * w.RB;  // row blocks of items, end to end: an equal share a block
    const long long w0 = (long long)blockIdx.x * work / gridDim.x, w1 = (long long)(blockIdx.x + 1) * work / gridDim.x;
    const float* sw = reinterpret_cast<const float*>(w.data + w.scale_off);
    bool waited = false;
    int acc[NB][4];
#pragma unroll
    for (int b = 0; b < NB; ++b)
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[b][i] = 0;

    for (long long at = w0; at < w1;) {
        cp_async_wait<0>();  // the last item's (empty) groups
        const int item = (int)(at / w.RB), rb0 = (int)(at - (long long)item * w.RB);
        const int rb1 = (int)min((long long)w.RB, rb0 + (w1 - at));
        at += rb1 - rb0;
        const int m0 = item * p.cols, rows = min(p.cols, c.a.M - m0);
        const int groups = (rb1 - rb0 + wr - 1) / wr;
        int left = rb0 + rw < rb1 ? ((rb1 - rb0 - rw + wr - 1) / wr) * nit : 0;
        int li = 0, lv = kw, ls = 0;
        const uint8_t* lp = w.data + (rb0 + rw) * rb_bytes + kw * kQcSeg + lane * 16;
        const long long lback = wr * rb_bytes - (long long)nit * wk * kQcSeg;
        const uint32_t to = smem_u32(ring) + lane * 16;
        auto load = [&]() {  // a group of copies, empty past the end, so that the groups' count is the ring's
            if (left > 0) {
                --left;
                if (lv < w.KS) {
                    const uint32_t d = to + ls * kQcSeg;
#pragma unroll
                    for (int i = 0; i < 4; ++i) cp_async16(d + 512 * i, lp + 512 * i);
                }
                lv += wk;
                lp += wk * kQcSeg;
                if (++li == nit) {
                    li = 0;
                    lv = kw;
                    lp += lback;
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
        __syncthreads();  // the last item's activations are no longer read
        if (!p.quant) stage_codes(sm, scale, p, m0, rows, tid, nthr);
        else if (c.a.xt == X_F32) stage_floats<X_F32>(sm, scale, top, p, m0, rows, tid, nthr);
        else if (c.a.xt == X_F16) stage_floats<X_F16>(sm, scale, top, p, m0, rows, tid, nthr);
        else stage_floats<X_BF16>(sm, scale, top, p, m0, rows, tid, nthr);
        __syncthreads();

        // this lane's columns (8 b + g) at offset xp, xq bytes from a tile to the next (0: it has no column)
        int xp[NB], xq[NB];
#pragma unroll
        for (int b = 0; b < NB; ++b) {
            const bool on = 8 * b + g < rows;
            xq[b] = on ? 64 : 0;
            xp[b] = on ? (8 * b + g) * p.pitch + t * 16 : p.off_zero;
        }
        int crb = rb0 + rw, cs = 0;  // row block, ring place
        for (int gi = 0; gi < groups; ++gi, crb += wr, flip ^= 1) {
            if (crb >= rb1) continue;
            int v = kw, xo[NB];
#pragma unroll
            for (int b = 0; b < NB; ++b) xo[b] = xp[b] + kw * 2 * xq[b];
            for (int ci = 0; ci < nit; ++ci, v += wk) {
                cp_async_wait<kDepth - 2>();
                __syncwarp();  // every lane's copies of this segment have landed, and the last one has been read
                load();
                const uint8_t* sp = ring + cs * kQcSeg + lane * 16;
                cs = cs + 1 == kDepth ? 0 : cs + 1;
                if (v < w.KS) {
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
                }
#pragma unroll
                for (int b = 0; b < NB; ++b) xo[b] += wk * 2 * xq[b];
            }
            // the row block's sums
            int* mine = red + (flip * (nthr / 32) + warp) * kRed;
#pragma unroll
            for (int b = 0; b < NB; ++b) {
                const int col = 8 * b + 2 * t;
                if (col < rows) {
                    mine[col * 16 + g] = acc[b][0];
                    mine[col * 16 + g + 8] = acc[b][2];
                }
                if (col + 1 < rows) {
                    mine[(col + 1) * 16 + g] = acc[b][1];
                    mine[(col + 1) * 16 + g + 8] = acc[b][3];
                }
                acc[b][0] = acc[b][1] = acc[b][2] = acc[b][3] = 0;
            }
            if (wk == 1) __syncwarp();
            else asm volatile("bar.sync %0, %1;" ::"r"(1 + rw), "r"(wk * 32) : "memory");
            const int* from = red + (flip * (nthr / 32) + rw * wk) * kRed;
            // the warps take turns at a short row block's sums
            for (int o = ((kw + gi) & (wk - 1)) * 32 + lane; o < rows * 16; o += wk * 32) {
                int sum = 0;
#pragma unroll 4
                for (int k2 = 0; k2 < wk; ++k2) sum += from[k2 * kRed + o];
                const int n = crb * 16 + (o & 15), r = o >> 4;
                if (n < w.N) x_store(c.y, c.yt, (long long)(m0 + r) * w.N + n, qc_scale(sum, __ldg(sw + n), scale[r], c.bias ? __ldg(c.bias + n) : 0.0f));
            }
        }
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
    auto fixed = [&](int cols, int warps) { return (long long)round_up(cols * 4, 16) + 16 + 2ll * warps * nb_of(cols) * 512 + (long long)warps * kDepth * kQcSeg; };
    double best = 0;
    for (int most : {8, 16, 32}) {
        int cols = c.a.M < most ? c.a.M : most;
        while (cols > 1 && (long long)cols * pl.pitch + fixed(cols, 8) > room) --cols;
        if ((long long)cols * pl.pitch + fixed(cols, 8) > room) continue;
        const int items = (c.a.M + cols - 1) / cols;
        cols = (c.a.M + items - 1) / items;
        const int nb = nb_of(cols);
        for (int warps : {16, 8}) {
            if ((long long)cols * pl.pitch + fixed(cols, warps) > room) continue;
            for (int wk = 1; wk <= warps; wk *= 2) {
                const int wr = warps / wk, nit = (w.KS + wk - 1) / wk;
                if (wr > 15 && wk > 1) continue;  // named barriers
                const long long work = (long long)items * w.RB, blocks = work < sms ? work : sms;
                const double share = (double)work / blocks;
                // segments a warp takes in turn and its row blocks' barriers and sums (about one each); an
                // item's staging
                const double cost = ceil(share / wr) * (nit + 1.0) * (warps / 8.0) * (nb == 1 ? 1.0 : nb == 2 ? 1.3 : 2.4) + (double)items / blocks * cols * w.KS * 0.1;
                if (best == 0 || cost < 0.999 * best || (cost <= 1.001 * best && nb <= pl.nb && wk > pl.wk)) {
                    best = cost;
                    pl.cols = cols;
                    pl.nb = nb;
                    pl.warps = warps;
                    pl.wk = wk;
                    pl.blocks = (int)blocks;
                    pl.items = items;
                }
            }
        }
    }
    if (best == 0) return pl;
    const long long act = (long long)pl.cols * pl.pitch;
    pl.off_zero = (int)act;
    pl.off_scale = pl.off_zero + 16;
    pl.off_red = pl.off_scale + round_up(pl.cols * 4, 16);
    pl.off_ring = pl.off_red + 2 * pl.warps * pl.nb * 512;
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
    p.wk = pl.wk;
    p.wr = pl.warps / pl.wk;
    p.wk_log2 = pl.wk == 1 ? 0 : pl.wk == 2 ? 1 : pl.wk == 4 ? 2 : pl.wk == 8 ? 3 : 4;
    p.pitch = pl.pitch;
    p.off_zero = pl.off_zero;
    p.off_scale = pl.off_scale;
    p.off_red = pl.off_red;
    p.off_ring = pl.off_ring;
    return pl.nb == 1 ? rows_go<1>(pl, p, smem_max, s) : pl.nb == 2 ? rows_go<2>(pl, p, smem_max, s) : rows_go<4>(pl, p, smem_max, s);
}

}  // namespace qmm
