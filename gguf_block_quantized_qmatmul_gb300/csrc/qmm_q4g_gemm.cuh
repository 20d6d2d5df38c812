// qmm_q4g_gemm.cuh -- products of 4-bit group-scale weights with many
// activation rows on tcgen05: prompts through a dense linear, and the
// experts' products of a batch (grouped by expert, any number of rows each).
//
// Mathematics.  Weight rows and activation rows are brought into f16's range
// by a power of two each (the weights' at layout time, the activations' by the
// preparation launch; f16 activations keep theirs), and
//   y = 2^-(a + b) sum_k f16(s 2^a (q - z)) (x 2^b).
// s 2^a and q - z are exact in f16, their product is rounded to 11 bits: half
// of the products (codes 0, +-1, 2, 4, 8 off the zero point) are exact, so the
// sum's error is below that of rounding an f16 result, and far below a bf16
// one.  bf16 activations are exact in f16 after scaling (values under 2^-29 of
// their row's largest lose bits).  f32 activations take two pieces of both
// operands, v = hi + lo, and three MMAs, hi hi + hi lo + lo hi: s (q - z) has
// at most 16 significant bits, so the weights' pieces are exact; the
// activations keep 22 bits.
//
// One persistent block per SM over units: 128 weight rows (8 row blocks, the
// MMA's M) x up to bx activation rows of one expert (its N, rounded up to 16).
//   warp 0      one thread: activation tiles (64 K, 128-byte swizzle), 2-D boxes; the
//               experts' rows were put in sorted order by the preparation launch
//               (gathering four rows a copy here measured 90 cycles a copy: 643 us
//               against the whole of 2048 tokens x 8 of 64 experts, 2048 -> 2 x 1024)
//   warp 1      one elected lane: four MMAs (twelve with two pieces) per 64 K, A in
//               tensor memory, B in shared memory
//   warp 2      raw weights: eight 1-D copies (a row block's two segments each)
//               per 256 K
//   warps 3-6   epilogue: accumulator columns to registers, scaled; the experts'
//               first product takes its up row from the lane eight away (paired
//               layout) for silu(g) u
//   warps 7-22  conversion: a lane's uint4 of codes becomes fragment registers
//               and goes to tensor memory as they are (16-lane x 128-bit
//               stores); four groups of four warps, one 64-K tile of a raw stage
//               each (a tile takes a group about 1400 cycles from end to end, and 192
//               rows' MMAs 384: with two groups those waited for it)
// The weights are bound for tensor memory, so shared memory feeds only the
// activation tiles to the MMAs.  With two pieces the tensor core's truncating
// f32 accumulation would show: the accumulator is restarted every kQgChunk
// tiles and the epilogue adds the chunks in registers.  A dense call with fewer
// units than SMs is split over K as well, and a last launch adds the slices.
#pragma once

#include <type_traits>

#include "qmm_q4g_rows.cuh"

namespace qmm {

constexpr int kQgEpiWarps = 8, kQgConvWarps = 8;
constexpr int kQgEpiHalves = kQgEpiWarps / 4, kQgGroups = kQgConvWarps / 4;  // warps per TMEM lane quarter
constexpr int kQgEpi0 = 3, kQgConv0 = kQgEpi0 + kQgEpiWarps;
constexpr int kQgThreads = (kQgConv0 + kQgConvWarps) * 32;
constexpr int kQgBX1 = 192, kQgBX2 = 64;  // activation rows per tile, at most: one piece, two pieces
constexpr int kQgRawMax = 4, kQgStageMax = 8;
constexpr int kQgChunk = 4;      // 64-K tiles per accumulation chunk (two pieces)
constexpr int kQgMaxE = 512;     // experts of a grouped call

struct QgGemmParams {
    QgCall c;
    float* part;          // P_DOWN: [T top_k][N]
    const float* xs;      // 2^-b per activation row (experts: per sorted position); NULL: 1
    const float* wis;     // 2^-a per weight row, layout order
    unsigned* err;
    int xrows;            // rows of an activation plane (the lo plane follows)
    int bx, box, accw, mtiles, ntiles, kt, nraw, nstage, grid;
    int ks;               // K slices (dense): f32 partial outputs [ks][M][N]
    int off_raw, off_bar;
};

// 32 columns of 16 lanes from fragment registers: lane 4 g + t's registers 2 j, 2 j + 1 are column 4 j + t of lanes g, g + 8
__device__ __forceinline__ void tc_st_frag(uint32_t taddr, const uint32_t v[16]) {
    asm volatile(
        "tcgen05.st.sync.aligned.16x128b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(taddr),
        "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(v[8]), "r"(v[9]),
        "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15])
        : "memory");
}

// true in one lane of a converged warp
__device__ __forceinline__ bool elect_one() {
    uint32_t p;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(p));
    return p != 0;
}

// One 64-K tile h of a segment of one row block: fragment registers of its f16 weights (and their rests).
template <int NP, int NG>
__device__ __forceinline__ void qg_convert(const uint8_t* seg, int h, int lane, uint32_t magic, float m0, float m1, uint32_t hi[16], uint32_t lo[16]) {
    const uint4 q = *reinterpret_cast<const uint4*>(seg + h * kQgTile + lane * 16);
    const uint32_t word[4] = {q.x, q.y, q.z, q.w};
    const uint32_t* sw = reinterpret_cast<const uint32_t*>(seg + 2 * kQgTile + (lane >> 2) * (8 * NG));
    uint32_t zl = 0, zh = 0;
    __half2 s0, s1;
#pragma unroll
    for (int s = 0; s < 4; ++s) {
        if (s == 0 || (NG == 4 && s == 2)) {
            const int gi = NG == 1 ? 0 : NG == 2 ? h : 2 * h + (s >> 1);
            const uint2 v = *reinterpret_cast<const uint2*>(sw + 2 * gi);
            zl = qg_zero<false>(v.x, false);
            zh = qg_zero<false>(v.y, true);
            s0 = __float2half2_rn(qg_scale(v.x) * m0);
            s1 = __float2half2_rn(qg_scale(v.y) * m1);
        }
        uint32_t a[4];
        qg_codes<false>(word[s], magic, zl, zh, a);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const __half2 c = *reinterpret_cast<__half2*>(&a[i]);
            const __half2 sc = i & 1 ? s1 : s0;
            const __half2 p = __hmul2(c, sc);
            hi[4 * s + i] = *reinterpret_cast<const uint32_t*>(&p);
            if (NP == 2) {
                const __half2 r = __hfma2(c, sc, __hneg2(p));
                lo[4 * s + i] = *reinterpret_cast<const uint32_t*>(&r);
            }
        }
    }
}

// After the last use: waits for the copies of every stage still in flight.
__device__ __forceinline__ void qg_drain(const QgRing& r, bool wrapped, int n, uint64_t* bars, volatile int* flags, unsigned* err) {
    for (int q = 0; q < n; ++q)
        if (q < r.s || wrapped) mbar_drain(smem_u32(&bars[q]), q < r.s ? r.ph : r.ph ^ 1u, flags, err);
}

// a unit's place
struct QgUnit {
    int e, p0, n, nt;  // expert, first position (row of x in a dense call), activation rows, row tile
    int split, j0, j1; // K slice, its 64-K tiles
};

template <int NP, int NG>
__global__ void __launch_bounds__(kQgThreads, 1) q4g_gemm_kernel(const __grid_constant__ CUtensorMap tx, const QgGemmParams p) {
    extern __shared__ __align__(1024) uint8_t smraw[];
    uint8_t* sm = smraw + ((1024 - (smem_u32(smraw) & 1023)) & 1023);
    const QgCall& c = p.c;
    const QgWeights& w = c.w;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    uint64_t* bars = reinterpret_cast<uint64_t*>(sm + p.off_bar);
    uint64_t* full = bars;                         // activation tile landed and weight pieces in tensor memory
    uint64_t* empty = full + kQgStageMax;          // stage consumed by the MMAs (commit)
    uint64_t* r_full = empty + kQgStageMax;        // raw weights landed
    uint64_t* r_empty = r_full + kQgRawMax;        // raw stage converted
    uint64_t* acc_full = r_empty + kQgRawMax;      // accumulator complete (commit)
    uint64_t* acc_empty = acc_full + 2;            // accumulator read
    static_assert((2 * kQgStageMax + 2 * kQgRawMax + 4) * 8 <= 256, "mbarriers overlap the TMEM slot");
    uint32_t* tslot = reinterpret_cast<uint32_t*>(sm + p.off_bar + 256);
    volatile int* flags = reinterpret_cast<volatile int*>(sm + p.off_bar + 320);
    int* col_slot = reinterpret_cast<int*>(sm + p.off_bar + 512);             // [warps][kQgBX1]
    float* col_scale = reinterpret_cast<float*>(col_slot + kQgEpiWarps * kQgBX1);  // [warps][kQgBX1]
    int* ts = reinterpret_cast<int*>(col_scale + kQgEpiWarps * kQgBX1);       // [E + 1] activation tiles before each expert
    const bool grouped = c.op != P_DENSE;
    const int slots = grouped ? c.r.T * c.r.top_k : c.M;
    if (tid == 0) {
        for (int i = 0; i < kQgStageMax; ++i) {
            mbar_init(smem_u32(&full[i]), 1 + 4);
            mbar_init(smem_u32(&empty[i]), 1);
        }
        for (int i = 0; i < kQgRawMax; ++i) {
            mbar_init(smem_u32(&r_full[i]), 1);
            mbar_init(smem_u32(&r_empty[i]), kQgConvWarps);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(smem_u32(&acc_full[i]), 1);
            mbar_init(smem_u32(&acc_empty[i]), kQgEpiWarps);
        }
        flags[0] = 0;
        fence_mbar_init();
    }
    if (warp == 1) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(tslot)), "n"(kTcTmemCols)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    grid_dep_launch();
    if (grouped) grid_dep_wait();
    if (warp == 0) {
        if (grouped) {
            const int per = (w.E + 31) / 32;
            int mine = 0;
            for (int i = 0; i < per; ++i) {
                const int e = lane * per + i;
                if (e < w.E) mine += (max(min(c.r.offsets[e + 1], slots) - max(c.r.offsets[e], 0), 0) + p.bx - 1) / p.bx;
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
                pre += (max(min(c.r.offsets[e + 1], slots) - max(c.r.offsets[e], 0), 0) + p.bx - 1) / p.bx;
            }
        } else if (lane == 0) {
            ts[0] = 0;
            ts[1] = p.mtiles;
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tslot;
    const int tiles_all = ts[w.E] * p.ntiles, units = tiles_all * p.ks;
    auto place = [&](int u) {
        QgUnit un;
        un.split = u / tiles_all;
        u -= un.split * tiles_all;
        const int nr = (w.KS + 1) / 2;  // raw stages
        un.j0 = 4 * (int)((long long)un.split * nr / p.ks);
        un.j1 = min(p.kt, 4 * (int)((long long)(un.split + 1) * nr / p.ks));
        const int st = u / p.ntiles;
        un.nt = u - st * p.ntiles;
        int lo = 0, hi = w.E;  // ts[lo] <= st < ts[hi]
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (ts[mid] <= st) lo = mid;
            else hi = mid;
        }
        un.e = lo;
        const int first = grouped ? max(c.r.offsets[lo], 0) : 0;
        const int end = grouped ? min(c.r.offsets[lo + 1], slots) : c.M;
        // an expert's rows in tiles of one size (a multiple of 16), not full ones and a rest
        const int tiles = ts[lo + 1] - ts[lo];
        const int size = ((end - first + tiles - 1) / tiles + 15) & ~15;
        un.p0 = first + (st - ts[lo]) * size;
        un.n = min(size, end - un.p0);
        return un;
    };
    if (!grouped && warp != 2) grid_dep_wait();  // weights are constant: their copies may start at once
    const int piece = p.bx * 128;
    auto stage = [&](int s) { return sm + s * NP * piece; };
    const int seg_bytes = qg_seg_bytes(NG);
    auto raw = [&](int s) { return sm + p.off_raw + s * 16 * seg_bytes; };

    if (warp == 0) {
        // ------------------------------ activations ------------------------------
        if (lane == 0) {
            QgRing g;
            bool ok = true, wrapped = false;
            for (int u = blockIdx.x; u < units && ok; u += gridDim.x) {
                const QgUnit un = place(u);
                const int boxes = (un.n + p.box - 1) / p.box;
                for (int j = un.j0; j < un.j1; ++j) {
                    if (!(ok = qg_wait(smem_u32(&empty[g.s]), g.ph ^ 1u, flags, p.err))) break;
                    const uint32_t bar = smem_u32(&full[g.s]), to = smem_u32(stage(g.s));
                    mbar_arrive_tx(bar, (uint32_t)(NP * boxes * p.box * 128));
                    for (int i = 0; i < boxes; ++i) {
                        tma_2d(to + i * p.box * 128, &tx, j * 64, un.p0 + i * p.box, bar);
                        if (NP == 2) tma_2d(to + piece + i * p.box * 128, &tx, j * 64, p.xrows + un.p0 + i * p.box, bar);
                    }
                    g.next(p.nstage);
                    wrapped |= g.s == 0;
                }
            }
            // let every copy land before the block can exit
            qg_drain(g, wrapped, p.nstage, full, flags, p.err);
        }
    } else if (warp == 1) {
        // ------------------------------ MMA issuer ------------------------------
        // The whole warp runs the loop, so that its values are uniform, and one elected lane
        // issues: inside a one-lane branch every MMA's operands take detours to uniform
        // registers (58 cycles an MMA and 410 a tile, against 128 cycles of MMAs at 64 rows).
        const bool lead = elect_one();
        const uint64_t d0 = tc_sdesc128(smem_u32(stage(0)));
        const uint32_t lo0 = (uint32_t)d0, dhi = (uint32_t)(d0 >> 32);
        QgRing g;
        int cc = 0, last = -1;  // accumulator uses; the last stage issued
        uint32_t last_ph = 0;
        bool ok = true;
        uint32_t ready = 0;
        for (int u = blockIdx.x; u < units && ok; u += gridDim.x) {
            const QgUnit un = place(u);
            const uint32_t idesc = tc_idesc((un.n + 15) / 16 * 16);
            const int chunk = NP == 2 ? kQgChunk : p.kt;
            for (int c0 = un.j0; c0 < un.j1 && ok; c0 += chunk, ++cc) {
                const int ab = cc & 1, use = cc >> 1;
                if (use > 0) ok = qg_wait(smem_u32(&acc_empty[ab]), (uint32_t)((use - 1) & 1), flags, p.err);
                if (!ok) break;
                tc_fence_after();
                const uint32_t dt = tmem + (uint32_t)(ab * p.accw);
                const int n = min(chunk, un.j1 - c0);
                for (int i = 0; i < n; ++i) {
                    const int s = g.s;
                    const uint32_t ph = g.ph;
                    g.next(p.nstage);
                    const uint32_t nxt = mbar_test(smem_u32(&full[g.s]), g.ph);
                    if (!ready) ok = qg_wait(smem_u32(&full[s]), ph, flags, p.err);
                    if (!ok) break;
                    tc_fence_after();
                    const uint32_t xhi = lo0 + (uint32_t)((s * NP * piece) >> 4), xlo = xhi + (uint32_t)(piece >> 4);
                    const uint32_t whi = tmem + (uint32_t)(2 * p.accw + 32 * NP * s), wlo = whi + 32;
                    __syncwarp();
                    if (lead) {
#pragma unroll
                        for (int pass = 0; pass < 2 * NP - 1; ++pass) {
                            const uint32_t wa = pass == 2 ? wlo : whi, xb = pass == 1 ? xlo : xhi;
#pragma unroll
                            for (int kk = 0; kk < 4; ++kk)
                                tc_mma(dt, wa + 8 * kk, ((uint64_t)dhi << 32) | (xb + 2 * kk), idesc, (i | pass | kk) != 0 ? 1u : 0u);
                        }
                        tc_commit(smem_u32(&empty[s]));
                    }
                    last = s;
                    last_ph = ph;
                    ready = nxt;
                }
                if (!ok) break;
                if (lead) tc_commit(smem_u32(&acc_full[ab]));
            }
        }
        // the last commits must land before tensor memory is released
        if (last >= 0) mbar_drain(smem_u32(&empty[last]), last_ph, flags, p.err);
    } else if (warp == 2) {
        // ------------------------------ raw weights ------------------------------
        QgRing r;
        bool ok = true, wrapped = false;
        for (int u = blockIdx.x; u < units && ok; u += gridDim.x) {
            const QgUnit un = place(u);
            const int nrb = min(8, w.RB - 8 * un.nt);
            const uint8_t* src = w.data + (long long)un.e * w.expert_stride + ((long long)(8 * un.nt + lane) * w.KS) * seg_bytes;
            for (int j = un.j0 / 4; 4 * j < un.j1; ++j) {
                const int s = r.s;
                if (!(ok = qg_wait(smem_u32(&r_empty[s]), r.ph ^ 1u, flags, p.err))) break;
                const int nseg = min(2, w.KS - 2 * j);
                const uint32_t bar = smem_u32(&r_full[s]);
                if (lane == 0) mbar_arrive_tx(bar, (uint32_t)(nrb * nseg * seg_bytes));
                __syncwarp();
                if (lane < nrb) bulk_g2s(smem_u32(raw(s)) + lane * 2 * seg_bytes, src + (long long)(2 * j) * seg_bytes, (uint32_t)(nseg * seg_bytes), bar);
                __syncwarp();
                r.next(p.nraw);
                wrapped |= r.s == 0;
            }
        }
        if (lane == 0) qg_drain(r, wrapped, p.nraw, r_full, flags, p.err);
    } else if (warp < kQgConv0) {
        // ------------------------------ epilogue ------------------------------
        const int ew = warp - kQgEpi0, q = warp & 3, half = ew >> 2;  // column chunks half, half + kQgEpiHalves, ...
        const uint32_t tq = (uint32_t)(32 * q) << 16;
        int* my_slot = col_slot + ew * kQgBX1;
        float* my_scale = col_scale + ew * kQgBX1;
        int cc = 0;
        bool ok = true;
        const int chunk = NP == 2 ? kQgChunk : p.kt;
        const int F = w.N / 2;
        for (int u = blockIdx.x; u < units && ok; u += gridDim.x) {
            const QgUnit un = place(u);
            const int nch = (un.n + 15) / 16;
            const int rb = 8 * un.nt + 2 * q + (lane >> 4);
            const int n = rb < w.RB ? qg_row(w, rb, lane & 15) : -1;
            const float wsn = rb < w.RB ? __ldg(p.wis + ((long long)un.e * w.RB + rb) * 16 + (lane & 15)) : 0.0f;
            __syncwarp();
            for (int col = lane; col < 16 * nch; col += 32) {
                int slot = -1;
                float xsc = 0.0f;
                if (col < un.n) {
                    slot = un.p0 + col;
                    if (grouped) {
                        slot = c.r.order[slot];
                        if (slot >= slots) slot = -1;
                    }
                    xsc = p.xs ? __ldcg(p.xs + un.p0 + col) : 1.0f;
                }
                my_slot[col] = slot;
                my_scale[col] = xsc;
            }
            __syncwarp();
            const float wup = __shfl_xor_sync(0xffffffffu, wsn, 8);  // the paired row's factor
            auto put_as = [&](auto* y, int k, const float v[16]) {  // columns 16 k..
                using Y = typename std::remove_pointer<decltype(y)>::type;
                if (c.op == P_GATE_UP) {
                    // lanes r < 8 have gate rows, r + 8 their up rows; each finishes one of two columns
                    const bool up = (lane & 8) != 0;
                    const int f = rb * 8 + (lane & 7);
                    const bool on = rb < w.RB && f < F;
#pragma unroll
                    for (int i = 0; i < 16; i += 2) {
                        const float got = __shfl_xor_sync(0xffffffffu, up ? v[i] : v[i + 1], 8);
                        const int col = 16 * k + i + (up ? 1 : 0);
                        const int slot = my_slot[col];
                        const float xsc = my_scale[col];
                        const float mine = (up ? v[i + 1] : v[i]) * wsn * xsc, theirs = got * wup * xsc;
                        const float r = NP == 2 ? swiglu(up ? theirs : mine, up ? mine : theirs) : swiglu_fast(up ? theirs : mine, up ? mine : theirs);
                        if (on && slot >= 0) y[(long long)slot * F + f] = to_type<Y>(r);
                    }
                } else if (n >= 0) {
#pragma unroll
                    for (int i = 0; i < 16; ++i) {
                        const int slot = my_slot[16 * k + i];
                        const float r = v[i] * wsn * my_scale[16 * k + i];
                        if (slot >= 0) y[(long long)slot * w.N + n] = to_type<Y>(r);
                    }
                }
            };
            auto put = [&](int k, const float v[16]) {
                if (c.op == P_DOWN || p.ks > 1) put_as(p.part + (long long)un.split * c.M * w.N, k, v);
                else if (NP == 2) put_as(static_cast<float*>(c.y), k, v);
                else if (c.xt == X_F16) put_as(static_cast<__half*>(c.y), k, v);
                else put_as(static_cast<__nv_bfloat16*>(c.y), k, v);
            };
            constexpr int kSums = kQgBX2 / 16 / kQgEpiHalves;
            float sum[NP == 2 ? kSums : 1][16];
            for (int c0 = un.j0; c0 < un.j1; c0 += chunk, ++cc) {
                const int ab = cc & 1, use = cc >> 1;
                if (!(ok = qg_wait(smem_u32(&acc_full[ab]), (uint32_t)(use & 1), flags, p.err))) break;
                tc_fence_after();
                __syncwarp();
                const uint32_t acol = tmem + tq + (uint32_t)(ab * p.accw);
                if (NP == 2) {
#pragma unroll
                    for (int k = 0; k < kSums; ++k) {
                        uint32_t r[16];
                        if (half + kQgEpiHalves * k < nch) {
                            tc_ld16(acol + 16 * (half + kQgEpiHalves * k), r);
                            tc_wait_ld();
#pragma unroll
                            for (int i = 0; i < 16; ++i) sum[NP == 2 ? k : 0][i] = c0 == un.j0 ? __uint_as_float(r[i]) : sum[NP == 2 ? k : 0][i] + __uint_as_float(r[i]);
                        }
                    }
                } else {
                    uint32_t r[16];
                    if (half < nch) tc_ld16(acol + 16 * half, r);
                    for (int k = half; k < nch; k += kQgEpiHalves) {
                        tc_wait_ld();
                        float v[16];
#pragma unroll
                        for (int i = 0; i < 16; ++i) v[i] = __uint_as_float(r[i]);
                        if (k + kQgEpiHalves < nch) tc_ld16(acol + 16 * (k + kQgEpiHalves), r);
                        put(k, v);
                    }
                }
                __syncwarp();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(smem_u32(&acc_empty[ab]));
            }
            if (!ok) break;
            if (NP == 2) {
#pragma unroll
                for (int k = 0; k < kSums; ++k)
                    if (half + kQgEpiHalves * k < nch) put(half + kQgEpiHalves * k, sum[NP == 2 ? k : 0]);
            }
        }
    } else {
        // ------------------------------ conversion ------------------------------
        const int cw = warp - kQgConv0, q = warp & 3, grp = cw >> 2;
        QgRing g, r;  // of the raw stage's first tile; of raw stages
        int count = 0;  // tiles before this raw stage
        const uint32_t magic = opaque(0x64006400u);
        bool ok = true;
        for (int u = blockIdx.x; u < units && ok; u += gridDim.x) {
            const QgUnit un = place(u);
            float m[2][2];  // 2^a of rows g, g + 8 of this warp's two row blocks
#pragma unroll
            for (int hh = 0; hh < 2; ++hh) {
                const int rb = min(8 * un.nt + 2 * q + hh, w.RB - 1);
                const float* is = p.wis + ((long long)un.e * w.RB + rb) * 16 + (lane >> 2);
                m[hh][0] = __frcp_rn(__ldg(is));
                m[hh][1] = __frcp_rn(__ldg(is + 8));
            }
            for (int j = un.j0; j < un.j1; j += 4) {
                const int rs = r.s, n = min(4, un.j1 - j);
                if (!(ok = qg_wait(smem_u32(&r_full[rs]), r.ph, flags, p.err))) break;
                r.next(p.nraw);
                // The groups take tiles in turn, whatever a unit's number of them: a group that waits
                // for the release of tile t - nstage has waited for t - groups - nstage, so that with
                // nstage >= groups the stage's barrier is at most one phase behind the wait's parity.
                for (int i = (grp - count) & (kQgGroups - 1); i < n; i += kQgGroups) {
                    QgRing at = g;
                    at.skip(i, p.nstage);
                    uint32_t hi[16], lo[16];
                    const uint8_t* seg = raw(rs) + 2 * q * 2 * seg_bytes + (i >> 1) * seg_bytes;
                    qg_convert<NP, NG>(seg, i & 1, lane, magic, m[0][0], m[0][1], hi, lo);
                    if (!(ok = qg_wait(smem_u32(&empty[at.s]), at.ph ^ 1u, flags, p.err))) break;
                    tc_fence_after();
                    __syncwarp();
                    const uint32_t col = tmem + ((uint32_t)(32 * q) << 16) + (uint32_t)(2 * p.accw + 32 * NP * at.s);
                    tc_st_frag(col, hi);
                    if (NP == 2) tc_st_frag(col + 32, lo);
                    qg_convert<NP, NG>(seg + 2 * seg_bytes, i & 1, lane, magic, m[1][0], m[1][1], hi, lo);
                    tc_st_frag(col + (16u << 16), hi);
                    if (NP == 2) tc_st_frag(col + (16u << 16) + 32, lo);
                    asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(smem_u32(&full[at.s]));
                }
                if (!ok) break;
                g.skip(n, p.nstage);
                count += n;
                __syncwarp();
                if (lane == 0) mbar_arrive(smem_u32(&r_empty[rs]));
            }
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "n"(kTcTmemCols) : "memory");
    }
}

}  // namespace qmm
