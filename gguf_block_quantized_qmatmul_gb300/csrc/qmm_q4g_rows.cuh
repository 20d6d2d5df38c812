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
// The kernel is bound by the weight stream (0.5 + 4 / G bytes a weight).  The
// work, items (a group of activation rows with their weight matrix) times row
// blocks, is dealt to one block an SM in equal contiguous shares.  Every warp
// has its own ring of kQgDepth segments in shared memory, filled by asynchronous
// 16-byte copies (each lane copies the codes that it will read); a tile of 16 rows x
// 64 K is then one conflict-free 16-byte load a lane, in fragment order, and
// about 9 (f16) or 11 (bf16) instructions turn a word of eight codes into MMA
// operands.  Measured at 1 x 28672 x 8192 (f16, G = 64): loads straight into
// registers, four segments ahead, 44 us (16 warps an SM, and waiting for the
// oldest load waited for younger ones too); one bulk copy per two segments 35
// us, and still 30 us with no arithmetic at all; these rings 28 us (4.5 TB/s,
// 62 % of the issue slots; groups of 64 keep 40 bytes a thread in local memory).  14336 x 4096 bf16 with 8 rows: 11.6 us, of which the
// launch and the staging of 64 KB of activations a block are some 4 (12.5 us with
// one staging load a thread in flight and a division an address); one row of
// 4096 x 4096 bf16: 5.4 us; 29 us for 16 tokens' second products of 8 of 128
// experts (768 -> 2048, G = 32), with the launch that adds a token's.  wk warps split a row block's K
// and add their sums through shared memory, one barrier among them per row block.
// Activations are staged once per item in the order the MMAs read them (16
// bytes a lane, conflict-free).  Weights are constant, so a dense call's first
// copies are issued before the grid it depends on has completed.
#pragma once

#include "qmm_q4g_internal.h"

namespace qmm {

constexpr int kQgDepth = 4;        // segments in a warp's ring
// warps per block, at most: more columns need more registers
__host__ __device__ constexpr int qg_row_warps(int nb) { return nb == 1 ? 24 : 16; }
constexpr int kQgRowMaxE = 512;    // experts whose items a block can look up
constexpr int kQgRowStatic = 4096; // the kernel's static arrays, rounded up

struct QgRowsParams {
    QgCall c;
    float* part;   // P_DOWN by expert: [T top_k][N]
    int by_slot, cols, np, wk, wk_log2, wr;
    int off_zero, off_red, off_ring;
};

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async4(uint32_t dst, const void* src) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

// (v & mask) | c in one instruction: c stays in a register (with two constants the compiler takes two)
template <uint32_t MASK>
__device__ __forceinline__ uint32_t and_or(uint32_t v, uint32_t c) {
    uint32_t d;
    asm("lop3.b32 %0, %1, %2, %3, 0xea;" : "=r"(d) : "r"(v), "n"(MASK), "r"(c));
    return d;
}
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
// (one less shift); bf16: 0x3D80 | q is 2^-4 + q 2^-11, so that these codes are
// (q - z) 2^-11: a group's sum of 128 products with up to 15 times an activation
// near the end of the f32 and bf16 range stays in that range (f16 activations
// do not reach it), and the rows' sums are multiplied by 2^11 at their end.
// zl, zh: the constants of rows g and g + 8 (qg_zero).
// magic: kQgMagic in a register.
template <bool BF>
constexpr uint32_t kQgMagic = BF ? 0x3D803D80u : 0x64006400u;
constexpr float kQgCodeUnit = 1.0f / 2048.0f;  // what a bf16 code's unit is
template <bool BF>
__device__ __forceinline__ void qg_codes(uint32_t w, uint32_t magic, uint32_t zl, uint32_t zh, uint32_t a[4]) {
    if (BF) {
        const __nv_bfloat162 l = *reinterpret_cast<__nv_bfloat162*>(&zl), h = *reinterpret_cast<__nv_bfloat162*>(&zh);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            uint32_t v = and_or<0x000f000fu>(w >> (4 * i), magic);
            const __nv_bfloat162 r = __hsub2(*reinterpret_cast<__nv_bfloat162*>(&v), i & 1 ? h : l);
            a[i] = *reinterpret_cast<const uint32_t*>(&r);
        }
    } else {
        const __half2 l = *reinterpret_cast<__half2*>(&zl), h = *reinterpret_cast<__half2*>(&zh);
        const __half2 sixteenth = __half2half2(__ushort_as_half(0x2C00));
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const uint32_t v = i ? w >> 8 : w;
            uint32_t lo = and_or<0x000f000fu>(v, magic), hi = and_or<0x00f000f0u>(v, magic);
            const __half2 r0 = __hsub2(*reinterpret_cast<__half2*>(&lo), l);
            const __half2 r1 = __hfma2(*reinterpret_cast<__half2*>(&hi), sixteenth, h);
            a[2 * i] = *reinterpret_cast<const uint32_t*>(&r0);
            a[2 * i + 1] = *reinterpret_cast<const uint32_t*>(&r1);
        }
    }
}
// f16: 1024 + z for row g, -(64 + z) for row g + 8; bf16: 2^-4 + z 2^-11 for both
template <bool BF>
__device__ __forceinline__ uint32_t qg_zero(uint32_t sw, bool second) {
    const uint32_t z = sw & 15u;
    if (BF) return z * 0x00010001u | kQgMagic<true>;
    return second ? (z * 0x00100010u) + 0xD400D400u : (z * 0x00010001u | 0x64006400u);
}

// Staged activations: 32 K of a column are 64 bytes, thread t's 16 at 16 t (the
// words of K 2 t, 8 + 2 t, 16 + 2 t, 24 + 2 t and their successors); the columns
// of the same 32 K are next to each other, then the next 32 K.
//
// A quad of lanes has 32 K of a row, 8 each (words j = K 8 lane + 2 j): a 4 x 4
// transposition among them makes each lane's four words the ones it stores.
__device__ __forceinline__ uint4 qg_quad_transpose(uint32_t w0, uint32_t w1, uint32_t w2, uint32_t w3, int lane) {
    const bool b0 = lane & 1, b1 = lane & 2;
    // lanes one apart: even ones keep words 0, 2 and take the partner's 0, 2
    uint32_t s0 = __shfl_xor_sync(0xffffffffu, b0 ? w0 : w1, 1), s1 = __shfl_xor_sync(0xffffffffu, b0 ? w2 : w3, 1);
    uint32_t x0 = b0 ? s0 : w0, x1 = b0 ? w1 : s0, y0 = b0 ? s1 : w2, y1 = b0 ? w3 : s1;
    // (x0, x1): word b0 of lanes 2 i, 2 i + 1; (y0, y1): word 2 + b0
    s0 = __shfl_xor_sync(0xffffffffu, b1 ? x0 : y0, 2);
    s1 = __shfl_xor_sync(0xffffffffu, b1 ? x1 : y1, 2);
    return b1 ? make_uint4(s0, s1, y0, y1) : make_uint4(x0, x1, s0, s1);
}

// Stage `rows` rows of x (row r at element offset at(r)) as columns of virtual segments v0..
// B 16-byte loads (f32: pairs of them) a thread are in flight.
template <int B, bool F32, class At>
__device__ __forceinline__ void qg_stage_as(uint8_t* sm, const void* x, int K, int KS, int rows, int np, int v0, At at, int tid, int nthr) {
    const int ncol = rows * np, n = KS * 4 * rows * 4;  // quads: (32 K, row)
    const uint32_t magic = 0xffffffffu / (uint32_t)rows + 1u;  // quad / rows = umulhi(quad, magic): quad rows < 2^32; 0 for one row
    for (int i0 = 0; i0 < n; i0 += B * nthr) {
        uint4 u[B][F32 ? 2 : 1];
        uint8_t* to[B];
#pragma unroll
        for (int b = 0; b < B; ++b) {
            const int i = i0 + b * nthr + tid, j = i & 3, quad = i >> 2;
            const int h = magic ? (int)__umulhi((uint32_t)quad, magic) : quad, r = quad - h * rows, k = 32 * h + 8 * j;
            const bool on = i < n && k < K;
            to[b] = i < n ? sm + ((size_t)(v0 * 4 + h) * ncol + r * np) * 64 + j * 16 : nullptr;
#pragma unroll
            for (int q = 0; q < (F32 ? 2 : 1); ++q) {
                u[b][q] = make_uint4(0u, 0u, 0u, 0u);
                if (on) u[b][q] = reinterpret_cast<const uint4*>(static_cast<const uint8_t*>(x) + (at(r) + k) * (F32 ? 4 : 2))[q];
            }
        }
#pragma unroll
        for (int b = 0; b < B; ++b) {
            const int i = i0 + b * nthr + tid, j = i & 3;
            if (i - (tid & 31) >= n) break;  // the whole warp is done
            if constexpr (F32) {
                float f[8] = {__uint_as_float(u[b][0].x), __uint_as_float(u[b][0].y), __uint_as_float(u[b][0].z), __uint_as_float(u[b][0].w),
                              __uint_as_float(u[b][1].x), __uint_as_float(u[b][1].y), __uint_as_float(u[b][1].z), __uint_as_float(u[b][1].w)};
#pragma unroll
                for (int pc = 0; pc < 3; ++pc) {
                    uint32_t w[4];
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        const uint32_t v = __float_as_uint(f[e]) & 0xffff0000u;
                        w[e >> 1] = e & 1 ? w[e >> 1] | v : v >> 16;
                        // the rest is exact; an infinity or NaN has none
                        f[e] = (v & 0x7f800000u) == 0x7f800000u ? 0.0f : f[e] - __uint_as_float(v);
                    }
                    const uint4 q = qg_quad_transpose(w[0], w[1], w[2], w[3], j);
                    if (i < n) *reinterpret_cast<uint4*>(to[b] + pc * 64) = q;
                }
            } else {
                const uint4 q = qg_quad_transpose(u[b][0].x, u[b][0].y, u[b][0].z, u[b][0].w, j);
                if (i < n) *reinterpret_cast<uint4*>(to[b]) = q;
            }
        }
    }
}
template <class At>
__device__ __forceinline__ void qg_stage(uint8_t* sm, const void* x, int xt, int K, int KS, int rows, int np, int v0, At at, int tid, int nthr) {
    if (xt == X_F32) qg_stage_as<2, true>(sm, x, K, KS, rows, np, v0, at, tid, nthr);
    else qg_stage_as<4, false>(sm, x, K, KS, rows, np, v0, at, tid, nthr);
}

constexpr int kQgMaxK = 32;  // slots of one token, at most

// TOK: P_DOWN with a token per item, whose experts' segments are taken end to end.
template <int NB, bool BF, int NG, bool TOK>
__global__ void __launch_bounds__(qg_row_warps(NB) * 32, 1) q4g_rows_kernel(const QgRowsParams p) {
    extern __shared__ __align__(16) uint8_t sm[];
    __shared__ int s_e[kQgMaxK];       // TOK: the token's experts (-1: skipped)
    __shared__ float s_wt[kQgMaxK];    // and their weights
    __shared__ int s_row[64];          // by expert: the columns' slots
    __shared__ int ts[kQgRowMaxE + 1]; // by expert: items before each
    const QgCall& c = p.c;
    const QgWeights& w = c.w;
    // the warp's index from one lane, so that what follows from it is known to be uniform
    const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31, g = lane >> 2, t = lane & 3, nthr = blockDim.x;
    const int wk = p.wk, wr = p.wr, kw = warp & (wk - 1), rw = warp >> p.wk_log2;
    constexpr int seg_bytes = qg_seg_bytes(NG), segk = 128 / NG;
    uint8_t* ring = sm + p.off_ring + warp * (kQgDepth * seg_bytes);
    const uint32_t magic = opaque(kQgMagic<BF>);
    if (tid == 0) *reinterpret_cast<uint4*>(sm + p.off_zero) = make_uint4(0u, 0u, 0u, 0u);  // what lanes without a column read
    grid_dep_launch();

    const int nex = TOK ? c.r.top_k : 1;
    const int VS = nex * w.KS;                             // virtual segments: TOK's experts end to end
    const int nit = (VS + wk - 1) >> p.wk_log2;            // segments per warp and row block
    const long long rb_bytes = (long long)w.KS * seg_bytes;
    const bool by_expert = c.op != P_DENSE && !p.by_slot;
    int items = c.op == P_DENSE ? (c.M + p.cols - 1) / p.cols : TOK ? c.r.T : c.r.T * c.r.top_k;
    if (by_expert) {
        grid_dep_wait();
        if (warp == 0) {
            // expert e has ceil(count / cols) items; lane l adds up experts l per.. l per + per
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
            if (lane == 31) ts[w.E] = pre;
            pre -= mine;
            for (int i = 0; i < per; ++i) {
                const int e = lane * per + i;
                if (e >= w.E) break;
                ts[e] = pre;
                pre += (max(min(c.r.offsets[e + 1], slots) - max(c.r.offsets[e], 0), 0) + p.cols - 1) / p.cols;
            }
        }
        __syncthreads();
        items = ts[w.E];
    }
    // this block's share: row blocks of items, end to end
    const long long work = (long long)items * w.RB;
    const long long w0 = (long long)blockIdx.x * work / gridDim.x, w1 = (long long)(blockIdx.x + 1) * work / gridDim.x;

    bool waited = by_expert;
    float acc[NB][4];
#pragma unroll
    for (int b = 0; b < NB; ++b)
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[b][i] = 0.0f;
    float* red = reinterpret_cast<float*>(sm + p.off_red);
    constexpr int kRed = NB * 128;  // sums of a warp: [column][16 rows]
    int flip = 0;                   // which of its two areas a row block's sums use

    for (long long at = w0; at < w1;) {
        cp_async_wait<0>();  // the last item's (empty) groups
        const int item = (int)(at / w.RB), rb0 = (int)(at - (long long)item * w.RB);
        const int rb1 = (int)min((long long)w.RB, rb0 + (w1 - at));
        at += rb1 - rb0;
        // the item: its experts and columns
        int rows = 1, expert = 0, first = 0;
        if (!waited && c.op != P_DENSE) {
            grid_dep_wait();
            waited = true;
        }
        if (TOK) {
            __syncthreads();  // the last item's experts are no longer read
            if (tid < nex) {
                const int slot = item * nex + tid;
                const int e = c.r.ids[slot];
                s_e[tid] = e >= 0 && e < w.E ? e : -1;
                s_wt[tid] = c.r.weights[slot];
            }
            __syncthreads();
        } else if (c.op == P_DENSE) {
            rows = min(p.cols, c.M - item * p.cols);
        } else if (p.by_slot) {
            expert = c.r.ids[item];
            if (expert < 0 || expert >= w.E) continue;
        } else {
            int lo = 0, hi = w.E;  // ts[lo] <= item < ts[hi]
            while (hi - lo > 1) {
                const int mid = (lo + hi) >> 1;
                if (ts[mid] <= item) lo = mid;
                else hi = mid;
            }
            expert = lo;
            const int slots = c.r.T * c.r.top_k, p0 = max(c.r.offsets[lo], 0), n = max(min(c.r.offsets[lo + 1], slots) - p0, 0);
            first = p0 + (item - ts[lo]) * p.cols;
            rows = min(p.cols, n - (item - ts[lo]) * p.cols);
        }
        const uint8_t* base = w.data + expert * w.expert_stride;
        const int groups = (rb1 - rb0 + wr - 1) / wr, total = rb0 + rw < rb1 ? ((rb1 - rb0 - rw + wr - 1) / wr) * nit : 0;
        // load cursor: virtual segment lv of row block lrb; this lane's bytes of it at lp; ring place ls
        int left = total, li = 0, lv = kw, ls = 0, lrb = rb0 + rw, lj = 0, lseg = kw;
        const uint8_t* lp = base + lrb * rb_bytes + kw * seg_bytes + lane * 16;
        const long long lback = wr * rb_bytes - (long long)nit * wk * seg_bytes;
        const uint32_t to = smem_u32(ring) + lane * 16;
        auto load = [&]() {  // a group of copies, empty past the end, so that the groups' count is the ring's
            if (left > 0) {
                --left;
                if (lv < VS) {
                    if (TOK) {
                        while (lseg >= w.KS) {
                            lseg -= w.KS;
                            ++lj;
                        }
                        lp = w.data + (long long)max(s_e[lj], 0) * w.expert_stride + lrb * rb_bytes + lseg * seg_bytes + lane * 16;
                    }
                    const uint32_t d = to + ls * seg_bytes;
                    cp_async16(d, lp);
                    cp_async16(d + kQgTile, lp + kQgTile);
                    if (lane < 4 * NG) cp_async16(d + 2 * kQgTile, lp + 2 * kQgTile);
                }
                lv += wk;
                if (TOK) lseg += wk;
                else lp += wk * seg_bytes;
                if (++li == nit) {
                    li = 0;
                    lv = kw;
                    if (TOK) {
                        lrb += wr;
                        lj = 0;
                        lseg = kw;
                    } else {
                        lp += lback;
                    }
                }
            }
            ls = ls + 1 == kQgDepth ? 0 : ls + 1;
            cp_async_commit();
        };
#pragma unroll
        for (int i = 0; i < kQgDepth - 1; ++i) load();
        if (!waited) {
            grid_dep_wait();
            waited = true;
        }
        __syncthreads();  // the last item's activations are no longer read
        if (by_expert) {
            if (tid < rows) {
                const int slot = c.r.order[first + tid];
                s_row[tid] = slot >= 0 && slot < c.r.T * c.r.top_k ? slot : 0;
            }
            __syncthreads();
        }
        const int ncol = rows * p.np;
        if (TOK) {
            for (int j = 0; j < nex; ++j)
                qg_stage(sm, c.x, c.xt, w.K, w.KS, 1, p.np, j * w.KS, [&](int) { return ((long long)item * nex + j) * c.ldx; }, tid, nthr);
        } else {
            qg_stage(sm, c.x, c.xt, w.K, w.KS, rows, p.np, 0, [&](int r) {
                const long long xr = c.op == P_DENSE ? (long long)item * p.cols + r
                                     : p.by_slot     ? (long long)item / c.r.top_k
                                     : c.op == P_GATE_UP ? (long long)s_row[r] / c.r.top_k
                                                         : (long long)s_row[r];
                return xr * c.ldx;
            }, tid, nthr);
        }
        __syncthreads();

        // this lane's columns (8 b + g) at offset xp, xq bytes from 32 K to the next (0: it has no column)
        int xp[NB], xq[NB];
#pragma unroll
        for (int b = 0; b < NB; ++b) {
            const bool on = 8 * b + g < ncol;
            xq[b] = on ? ncol * 64 : 0;
            xp[b] = on ? (8 * b + g) * 64 + t * 16 : p.off_zero;
        }
        int crb = rb0 + rw, cs = 0;  // row block, ring place
        for (int gi = 0; gi < groups; ++gi, crb += wr, flip ^= 1) {
            if (crb >= rb1) continue;
            int cj = 0, cseg = kw, v = kw;
            int xo[NB];
#pragma unroll
            for (int b = 0; b < NB; ++b) xo[b] = xp[b] + kw * 4 * xq[b];
            for (int ci = 0; ci < nit; ++ci, v += wk) {
                cp_async_wait<kQgDepth - 2>();
                __syncwarp();  // every lane's copies of this segment have landed, and the last one has been read
                load();
                const uint8_t* sp = ring + cs * seg_bytes;
                cs = cs + 1 == kQgDepth ? 0 : cs + 1;
                bool on = v < VS;
                float wt = 1.0f;
                if (TOK && on) {
                    while (cseg >= w.KS) {
                        cseg -= w.KS;
                        ++cj;
                    }
                    on = s_e[cj] >= 0;
                    wt = s_wt[cj];
                }
                if (TOK) cseg += wk;
                if (on) {
                    const uint4 c0 = reinterpret_cast<const uint4*>(sp)[lane], c1 = reinterpret_cast<const uint4*>(sp + kQgTile)[lane];
                    uint32_t sw[2 * NG];
                    const uint8_t* sq = sp + 2 * kQgTile + g * (8 * NG);
                    if (NG == 1) {
                        const uint2 u = *reinterpret_cast<const uint2*>(sq);
                        sw[0] = u.x;
                        sw[1] = u.y;
                    } else {
#pragma unroll
                        for (int i = 0; i < NG / 2; ++i) {
                            const uint4 u = reinterpret_cast<const uint4*>(sq)[i];
                            sw[4 * i] = u.x;
                            sw[4 * i + 1] = u.y;
                            sw[4 * i + 2] = u.z;
                            sw[4 * i + 3] = u.w;
                        }
                    }
                    float gr[NB][4];
                    uint32_t zl = 0, zh = 0;
#pragma unroll
                    for (int q4 = 0; q4 < 4; ++q4) {  // 32 K a step
                        const int gi4 = q4 * 32 / segk;
                        const uint32_t sw0 = sw[2 * gi4], sw1 = sw[2 * gi4 + 1];
                        const bool start = q4 * 32 % segk == 0;
                        if (start) {
                            zl = qg_zero<BF>(sw0, false);
                            zh = qg_zero<BF>(sw1, true);
                        }
                        const uint4 cw = q4 < 2 ? c0 : c1;
                        uint32_t a0[4], a1[4];
                        qg_codes<BF>(q4 & 1 ? cw.z : cw.x, magic, zl, zh, a0);
                        qg_codes<BF>(q4 & 1 ? cw.w : cw.y, magic, zl, zh, a1);
#pragma unroll
                        for (int b = 0; b < NB; ++b) {
                            const uint4 xv = *reinterpret_cast<const uint4*>(sm + xo[b] + q4 * xq[b]);
                            if (start) qg_mma<BF, true>(gr[b], a0, xv.x, xv.y);
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
#pragma unroll
                for (int b = 0; b < NB; ++b) xo[b] += wk * 4 * xq[b];
            }
            // the row block's sums
            float* mine = red + (flip * (nthr / 32) + warp) * kRed;
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
            }
            if (wk == 1) __syncwarp();
            else asm volatile("bar.sync %0, %1;" ::"r"(1 + rw), "r"(wk * 32) : "memory");
            const float* from = red + (flip * (nthr / 32) + rw * wk) * kRed;
            const int per_log2 = w.paired ? 3 : 4;  // rows of y per row block
            auto sum = [&](int r, int row) {
                float v2 = 0.0f;
                for (int pc = 0; pc < p.np; ++pc) {
                    const float* f = from + (r * p.np + pc) * 16 + row;
#pragma unroll 4
                    for (int k2 = 0; k2 < wk; ++k2) v2 += f[k2 * kRed];
                }
                return BF ? v2 * (1.0f / kQgCodeUnit) : v2;
            };
            // the warps take turns at a short row block's sums
            for (int o = ((kw + gi) & (wk - 1)) * 32 + lane; o < rows << per_log2; o += wk * 32) {
                const int row = o & ((1 << per_log2) - 1), r = o >> per_log2;
                const float v0 = sum(r, row);
                if (c.op == P_GATE_UP) {
                    const float u = sum(r, row + 8);
                    const int f = crb * 8 + row, F = w.N / 2;
                    const long long slot = p.by_slot ? (long long)item : (long long)s_row[r];
                    if (f < F) x_store(c.y, c.xt, slot * F + f, swiglu(v0, u));
                } else {
                    const int n = crb * 16 + row;
                    if (n < w.N) {
                        if (c.op == P_DENSE)
                            x_store(c.y, c.xt, ((long long)item * p.cols + r) * w.N + n, v0);
                        else if (TOK)
                            x_store(c.y, c.xt, (long long)item * w.N + n, v0);
                        else
                            p.part[(long long)s_row[r] * w.N + n] = v0;
                    }
                }
            }
        }
    }
    if (!waited) grid_dep_wait();
}

}  // namespace qmm
