// qmm_q4g_rows.cuh -- products of 4-bit group-scale weights with few
// activation rows: decode steps and the experts of a few tokens.
//
// Mathematics.  y[n] = sum_groups s (sum_k (q - z) x): the codes less their
// zero point are integers in -15..15, exact in f16 and bf16, so they are the
// A operand of a 16 x 8 x 16 warp MMA as they are; a group's products
// accumulate in f32 and enter the row's f32 sum with one FMA by the f32 scale.
// No weight is rounded.  Activations are the B operand in their own type
// (f16, bf16); an f32 value is its three bf16 pieces, 8 bits each by
// truncation (exact, and no overflow), in three columns whose sums are added
// at the end.
//
// The kernel is bound by the weight stream (0.5 + 4 / G bytes a weight).  A
// warp's tile of 16 rows x 64 K is one coalesced 512-byte load straight into
// the fragment registers (no shared memory, no shuffles): about 9 (f16) or 11
// (bf16) instructions per word of eight codes turn it into MMA operands.
// kQgDepth segments of 128 K per warp are in flight, across row blocks; a
// block's warps split K (wk) and row blocks, and add their sums through
// shared memory with one barrier per row block.  Activations are staged once
// per block in the order the MMAs read them (16 bytes a lane, conflict-free).
// Weights are constant, so a dense call's first loads are issued before the
// grid it depends on has completed.
#pragma once

#include "qmm_q4g_internal.h"

namespace qmm {

constexpr int kQgDepth = 4;

struct QgRowsParams {
    QgCall c;
    float* part;   // P_DOWN by expert: [T top_k][N]
    int by_slot, cols, np, wk, off_red;
};

// FIRST: d = A B, else d += A B
template <bool BF, bool FIRST>
__device__ __forceinline__ void qg_mma(float d[4], const uint32_t a[4], uint32_t b0, uint32_t b1) {
    if (BF && FIRST)
        asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};"
            : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
            : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.0f));
    else if (BF)
        asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
            : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
            : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
    else if (FIRST)
        mma_f16_z(d, a[0], a[1], a[2], a[3], b0, b1);
    else
        mma_f16(d, a[0], a[1], a[2], a[3], b0, b1);
}

// The eight codes of one word less their zero points, exact, as fragment
// registers.  f16: 0x6400 | q is 1024 + q and 0x6400 | q << 4 is 1024 + 16 q
// (one less shift); bf16: 0x4300 | q is 128 + q.  zl, zh: the constants of
// rows g and g + 8 (qg_zero).
template <bool BF>
__device__ __forceinline__ void qg_codes(uint32_t w, uint32_t zl, uint32_t zh, uint32_t a[4]) {
    if (BF) {
        const __nv_bfloat162 l = *reinterpret_cast<__nv_bfloat162*>(&zl), h = *reinterpret_cast<__nv_bfloat162*>(&zh);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            uint32_t v = ((w >> (4 * i)) & 0x000f000fu) | 0x43004300u;
            const __nv_bfloat162 r = __hsub2(*reinterpret_cast<__nv_bfloat162*>(&v), i & 1 ? h : l);
            a[i] = *reinterpret_cast<const uint32_t*>(&r);
        }
    } else {
        const __half2 l = *reinterpret_cast<__half2*>(&zl), h = *reinterpret_cast<__half2*>(&zh);
        const __half2 sixteenth = __half2half2(__ushort_as_half(0x2C00));
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const uint32_t v = i ? w >> 8 : w;
            uint32_t lo = (v & 0x000f000fu) | 0x64006400u, hi = (v & 0x00f000f0u) | 0x64006400u;
            const __half2 r0 = __hsub2(*reinterpret_cast<__half2*>(&lo), l);
            const __half2 r1 = __hfma2(*reinterpret_cast<__half2*>(&hi), sixteenth, h);
            a[2 * i] = *reinterpret_cast<const uint32_t*>(&r0);
            a[2 * i + 1] = *reinterpret_cast<const uint32_t*>(&r1);
        }
    }
}
// f16: 1024 + z for row g, -(64 + z) for row g + 8; bf16: 128 + z for both
template <bool BF>
__device__ __forceinline__ uint32_t qg_zero(uint32_t sw, bool second) {
    const uint32_t z = sw & 15u;
    if (BF) return z * 0x00010001u | 0x43004300u;
    return second ? (z * 0x00100010u) + 0xD400D400u : (z * 0x00010001u | 0x64006400u);
}

template <int NG>
struct QgSeg {
    uint4 c[2];
    uint32_t sw[2 * NG];
};

template <int NG>
__device__ __forceinline__ void qg_load(QgSeg<NG>& s, const uint8_t* p, int lane) {
    s.c[0] = __ldg(reinterpret_cast<const uint4*>(p) + lane);
    s.c[1] = __ldg(reinterpret_cast<const uint4*>(p + kQgTile) + lane);
    const uint8_t* q = p + 2 * kQgTile + (lane >> 2) * (8 * NG);
    if (NG == 1) {
        const uint2 v = __ldg(reinterpret_cast<const uint2*>(q));
        s.sw[0] = v.x;
        s.sw[1] = v.y;
    } else {
#pragma unroll
        for (int i = 0; i < NG / 2; ++i) {
            const uint4 v = __ldg(reinterpret_cast<const uint4*>(q) + i);
            s.sw[4 * i] = v.x;
            s.sw[4 * i + 1] = v.y;
            s.sw[4 * i + 2] = v.z;
            s.sw[4 * i + 3] = v.w;
        }
    }
}

// 16-bit words of columns in fragment order: K position k of virtual segment v
// of column c.  Per 32 K a column has 64 bytes, thread t's 16 at 16 t.
__device__ __forceinline__ uint32_t* qg_xword(uint8_t* sm, int ncol, int v, int col, int k) {
    const int h = k >> 5, s = (k >> 4) & 1, hi = (k >> 3) & 1, t = (k & 7) >> 1;
    return reinterpret_cast<uint32_t*>(sm + ((size_t)(v * 4 + h) * ncol + col) * 64 + t * 16 + (2 * s + hi) * 4);
}

// Stage one row of x as column(s) col.. of virtual segments v0..: eight values a step.
__device__ __forceinline__ void qg_stage(uint8_t* sm, const void* x, int xt, long long at, int K, int KS, int ncol, int v0, int col,
                                         int tid, int nthr) {
    for (int i = tid; i < KS * (kQgSegK / 8); i += nthr) {
        const int k = 8 * i;
        if (xt == X_F32) {
            float f[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) f[j] = 0.0f;
            if (k < K) {
                const float4 a = *reinterpret_cast<const float4*>(static_cast<const float*>(x) + at + k);
                const float4 b = *reinterpret_cast<const float4*>(static_cast<const float*>(x) + at + k + 4);
                f[0] = a.x; f[1] = a.y; f[2] = a.z; f[3] = a.w;
                f[4] = b.x; f[5] = b.y; f[6] = b.z; f[7] = b.w;
            }
#pragma unroll
            for (int pc = 0; pc < 3; ++pc) {
                uint32_t w[4];
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const uint32_t u = __float_as_uint(f[j]) & 0xffff0000u;
                    w[j >> 1] = j & 1 ? w[j >> 1] | u : u >> 16;
                    // the rest is exact; an infinity or NaN has none
                    f[j] = (u & 0x7f800000u) == 0x7f800000u ? 0.0f : f[j] - __uint_as_float(u);
                }
#pragma unroll
                for (int j = 0; j < 4; ++j) *qg_xword(sm, ncol, v0 + (k >> 7), col + pc, (k & 127) + 2 * j) = w[j];
            }
        } else {
            uint4 u = make_uint4(0u, 0u, 0u, 0u);
            if (k < K) u = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(x) + at + k);
            const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
            for (int j = 0; j < 4; ++j) *qg_xword(sm, ncol, v0 + (k >> 7), col, (k & 127) + 2 * j) = w[j];
        }
    }
}

constexpr int kQgMaxK = 32;  // slots of one token, at most

// TOK: P_DOWN with a token per item, whose experts' segments are taken end to end.
template <int NB, bool BF, int NG, bool TOK>
__global__ void __launch_bounds__(512) q4g_rows_kernel(const QgRowsParams p) {
    extern __shared__ __align__(16) uint8_t sm[];
    __shared__ int s_e[kQgMaxK];       // TOK: the token's experts (-1: skipped)
    __shared__ float s_wt[kQgMaxK];    // and their weights
    __shared__ int s_row[64];          // by expert: the columns' slots
    __shared__ int s_item[3];          // expert, first position, columns
    const QgCall& c = p.c;
    const QgWeights& w = c.w;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t = lane & 3, nthr = blockDim.x;
    const int wk = p.wk, wr = nthr / 32 / wk, kw = warp % wk, rw = warp / wk;
    constexpr int seg_bytes = qg_seg_bytes(NG), segk = 128 / NG;
    // this block's row blocks
    const int rb0 = (int)((long long)blockIdx.x * w.RB / gridDim.x), rb1 = (int)((long long)(blockIdx.x + 1) * w.RB / gridDim.x);
    const int nex = TOK ? c.r.top_k : 1;
    const int VS = nex * w.KS;                        // virtual segments
    const int nit = (VS + wk - 1) / wk;               // segments per warp and row block
    const int total = ((rb1 - rb0) + wr - 1) / wr * nit;

    grid_dep_launch();
    QgSeg<NG> st[kQgDepth];
    // load cursor: segment lv of row block lrb, at lp (TOK: expert lj, its segment lseg)
    int li = 0, lv = kw, lrb = rb0 + rw, lj = 0, lseg = kw;
    const long long row_bytes = (long long)w.KS * seg_bytes;
    const uint8_t* base = w.data;
    const uint8_t* lp = nullptr;
    auto load_start = [&]() { lp = base + lrb * row_bytes + kw * seg_bytes; };
    auto load = [&](int d) {
        if (lrb < rb1 && lv < VS) {
            if (TOK) {
                while (lseg >= w.KS) {
                    lseg -= w.KS;
                    ++lj;
                }
                lp = w.data + (long long)max(s_e[lj], 0) * w.expert_stride + lrb * row_bytes + lseg * seg_bytes;
            }
            qg_load<NG>(st[d], lp, lane);
        }
        lv += wk;
        if (TOK) lseg += wk;
        else lp += wk * seg_bytes;
        if (++li == nit) {
            li = 0;
            lv = kw;
            lrb += wr;
            if (TOK) {
                lj = 0;
                lseg = kw;
            } else {
                lp += wr * row_bytes - nit * wk * seg_bytes;
            }
        }
    };
    if (c.op == P_DENSE) {
        load_start();
#pragma unroll
        for (int d = 0; d < kQgDepth; ++d)
            if (d < total) load(d);
    }
    if (tid == 0) *reinterpret_cast<uint4*>(sm + p.off_red - 16) = make_uint4(0u, 0u, 0u, 0u);  // what lanes without a column read
    grid_dep_wait();

    // the item: its experts and columns
    int rows = 1;
    if (TOK) {
        if (tid < nex) {
            const int slot = (int)blockIdx.y * nex + tid;
            const int e = c.r.ids[slot];
            s_e[tid] = e >= 0 && e < w.E ? e : -1;
            s_wt[tid] = c.r.weights[slot];
        }
        __syncthreads();
    } else if (c.op == P_DENSE) {
        rows = min(p.cols, c.M - (int)blockIdx.y * p.cols);
    } else if (p.by_slot) {
        const int e = c.r.ids[blockIdx.y];
        if (e < 0 || e >= w.E) return;
        base = w.data + e * w.expert_stride;
    } else {
        if (warp == 0) {
            // expert e has ceil(count / cols) items; lane l takes experts l per.. l per + per
            const int per = (w.E + 31) / 32, slots = c.r.T * c.r.top_k;
            int mine = 0;
            for (int i = 0; i < per; ++i) {
                const int e = lane * per + i;
                if (e < w.E) mine += (max(min(c.r.offsets[e + 1], slots) - max(c.r.offsets[e], 0), 0) + p.cols - 1) / p.cols;
            }
            int pre = mine;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int u = __shfl_up_sync(0xffffffffu, pre, o);
                if (lane >= o) pre += u;
            }
            if (lane == 31 && (int)blockIdx.y >= pre) s_item[0] = -1;
            pre -= mine;
            if ((int)blockIdx.y >= pre && (int)blockIdx.y < pre + mine)
                for (int i = 0; i < per; ++i) {
                    const int e = lane * per + i;
                    if (e >= w.E) break;
                    const int p0 = max(c.r.offsets[e], 0), n = max(min(c.r.offsets[e + 1], slots) - p0, 0);
                    const int items = (n + p.cols - 1) / p.cols, at = (int)blockIdx.y - pre;
                    if (at >= 0 && at < items) {
                        s_item[0] = e;
                        s_item[1] = p0 + at * p.cols;
                        s_item[2] = min(p.cols, n - at * p.cols);
                    }
                    pre += items;
                }
        }
        __syncthreads();
        if (s_item[0] < 0) return;
        rows = s_item[2];
        base = w.data + s_item[0] * w.expert_stride;
        if (tid < rows) {
            const int slot = c.r.order[s_item[1] + tid];
            s_row[tid] = slot >= 0 && slot < c.r.T * c.r.top_k ? slot : 0;
        }
    }
    if (c.op != P_DENSE) {
        load_start();
#pragma unroll
        for (int d = 0; d < kQgDepth; ++d)
            if (d < total) load(d);
        if (!p.by_slot) __syncthreads();  // the slots
    }
    // activations
    const int ncol = rows * p.np;
    if (TOK) {
        for (int j = 0; j < nex; ++j)
            qg_stage(sm, c.x, c.xt, ((long long)blockIdx.y * nex + j) * c.ldx, w.K, w.KS, ncol, j * w.KS, 0, tid, nthr);
    } else {
        for (int r = 0; r < rows; ++r) {
            const long long xr = c.op == P_DENSE ? (long long)blockIdx.y * p.cols + r
                                 : p.by_slot     ? (long long)blockIdx.y / c.r.top_k
                                 : c.op == P_GATE_UP ? (long long)s_row[r] / c.r.top_k
                                                     : (long long)s_row[r];
            qg_stage(sm, c.x, c.xt, xr * c.ldx, w.K, w.KS, ncol, 0, r * p.np, tid, nthr);
        }
    }
    __syncthreads();

    float acc[NB][4];
#pragma unroll
    for (int b = 0; b < NB; ++b)
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[b][i] = 0.0f;
    float* red = reinterpret_cast<float*>(sm + p.off_red);
    constexpr int kRed = NB * 128;  // sums of a warp: [column][16 rows]
    // compute cursor; this lane's columns (8 b + g) at offset xp, xq bytes from 32 K to the next (0: it has no column)
    int ci = 0, cr = 0, cv = kw, crb = rb0 + rw, cj = 0, cseg = kw;
    int xp[NB], xq[NB];
#pragma unroll
    for (int b = 0; b < NB; ++b) {
        const bool on = 8 * b + g < ncol;
        xq[b] = on ? ncol * 64 : 0;
        xp[b] = on ? kw * 4 * xq[b] + (8 * b + g) * 64 + t * 16 : p.off_red - 16;
    }
    for (int it = 0; it < total; it += kQgDepth) {
#pragma unroll
        for (int d = 0; d < kQgDepth; ++d) {
            if (it + d >= total) break;
            if (crb < rb1 && cv < VS) {
                float wt = 1.0f;
                bool on = true;
                if (TOK) {
                    while (cseg >= w.KS) {
                        cseg -= w.KS;
                        ++cj;
                    }
                    on = s_e[cj] >= 0;
                    wt = s_wt[cj];
                }
                if (on) {
                    float gr[NB][4];
#pragma unroll
                    for (int q4 = 0; q4 < 4; ++q4) {  // 32 K a step
                        const int gi = q4 * 32 / segk;
                        const uint32_t sw0 = st[d].sw[2 * gi], sw1 = st[d].sw[2 * gi + 1];
                        const uint32_t zl = qg_zero<BF>(sw0, false), zh = qg_zero<BF>(sw1, true);
                        const uint4 cw = st[d].c[q4 >> 1];
                        uint32_t a0[4], a1[4];
                        qg_codes<BF>(q4 & 1 ? cw.z : cw.x, zl, zh, a0);
                        qg_codes<BF>(q4 & 1 ? cw.w : cw.y, zl, zh, a1);
                        const bool first = q4 * 32 % segk == 0;
#pragma unroll
                        for (int b = 0; b < NB; ++b) {
                            const uint4 xv = *reinterpret_cast<const uint4*>(sm + xp[b] + q4 * xq[b]);
                            if (first) qg_mma<BF, true>(gr[b], a0, xv.x, xv.y);
                            else qg_mma<BF, false>(gr[b], a0, xv.x, xv.y);
                            qg_mma<BF, false>(gr[b], a1, xv.z, xv.w);
                        }
                        if ((q4 + 1) * 32 % segk == 0) {  // the group's end
                            const float s0 = TOK ? qg_scale(sw0) * wt : qg_scale(sw0), s1 = TOK ? qg_scale(sw1) * wt : qg_scale(sw1);
#pragma unroll
                            for (int b = 0; b < NB; ++b) {
                                acc[b][0] = fmaf(s0, gr[b][0], acc[b][0]);
                                acc[b][1] = fmaf(s0, gr[b][1], acc[b][1]);
                                acc[b][2] = fmaf(s1, gr[b][2], acc[b][2]);
                                acc[b][3] = fmaf(s1, gr[b][3], acc[b][3]);
                            }
                        }
                    }
                }
            }
            if (it + d + kQgDepth < total) load(d);
            cv += wk;
            if (TOK) cseg += wk;
#pragma unroll
            for (int b = 0; b < NB; ++b) xp[b] += wk * 4 * xq[b];
            if (++ci == nit) {  // the row block's sums
                float* mine = red + ((cr & 1) * (nthr / 32) + warp) * kRed;
#pragma unroll
                for (int b = 0; b < NB; ++b) {
                    const int col = 8 * b + 2 * t;
                    if (col < ncol) {
                        mine[col * 16 + g] = acc[b][0];
                        mine[col * 16 + g + 8] = acc[b][2];
                    }
                    if (col + 1 < ncol) {
                        mine[(col + 1) * 16 + g] = acc[b][1];
                        mine[(col + 1) * 16 + g + 8] = acc[b][3];
                    }
                    acc[b][0] = acc[b][1] = acc[b][2] = acc[b][3] = 0.0f;
                    xp[b] -= nit * wk * 4 * xq[b];
                }
                __syncthreads();
                if (crb < rb1) {
                    const float* from = red + ((cr & 1) * (nthr / 32) + rw * wk) * kRed;
                    const int per = w.paired ? 8 : 16;
                    auto sum = [&](int r, int row) {
                        float v2 = 0.0f;
                        for (int pc = 0; pc < p.np; ++pc) {
                            const float* f = from + (r * p.np + pc) * 16 + row;
#pragma unroll 4
                            for (int k2 = 0; k2 < wk; ++k2) v2 += f[k2 * kRed];
                        }
                        return v2;
                    };
                    // the warps take turns at a short row block's sums
                    for (int o = ((kw + cr) & (wk - 1)) * 32 + lane; o < per * rows; o += wk * 32) {
                        const int row = o % per, r = o / per;
                        const float v0 = sum(r, row);
                        if (c.op == P_GATE_UP) {
                            const float u = sum(r, row + 8);
                            const int f = crb * 8 + row, F = w.N / 2;
                            const long long slot = p.by_slot ? (long long)blockIdx.y : (long long)s_row[r];
                            if (f < F) x_store(c.y, c.xt, slot * F + f, swiglu(v0, u));
                        } else {
                            const int n = crb * 16 + row;
                            if (n < w.N) {
                                if (c.op == P_DENSE)
                                    x_store(c.y, c.xt, ((long long)blockIdx.y * p.cols + r) * w.N + n, v0);
                                else if (TOK)
                                    x_store(c.y, c.xt, (long long)blockIdx.y * w.N + n, v0);
                                else
                                    p.part[(long long)s_row[r] * w.N + n] = v0;
                            }
                        }
                    }
                }
                ci = 0;
                ++cr;
                cv = kw;
                crb += wr;
                if (TOK) {
                    cj = 0;
                    cseg = kw;
                }
            }
        }
    }
}

}  // namespace qmm
