// qmm_q8c_gemm.cu -- 8-bit channel-scaled products of many activation rows on
// tcgen05.
//
// Mathematics.  sm_103a's tensor cores multiply 8-bit integers at a twelfth of
// their f16 rate (warp MMAs) or not at all (tcgen05), so the codes become f16,
// exactly, and their products are added in f32.  A sum of integers is exact
// there while no partial sum passes 2^24, and by Cauchy and Schwarz none does
// where (sum of squares of a weight row)(sum of squares of an activation row) <
// 2^48: the weights' largest sum of squares is in their layout, the
// activations' are computed with their codes.  Rows as models have them (sigma
// about 30 codes, 16384 K) fulfil it and are accumulated in one go.  In a call
// where some row does not, the accumulator is restarted every 1024 K (1024 x
// 2^14 = 2^24: at most 127 x 128 a product of quantized activations; given codes
// of -128 twice reach 2^24 itself, which f32 holds) and the parts are added as
// integers.  So y is the same as the row kernel's, bit for bit.
//
// The structure is the 4-bit GEMM's (qmm_q4g_gemm.cuh): one persistent block an
// SM, pairs of blocks (cta_group::2) on 256 weight rows x up to 256 activation
// rows; converted weights are the A operand in tensor memory, activations come
// by TMA in 128-byte swizzled tiles.  27 warps' roles:
//   warp 0      activation tiles, 128 K each (256 for up to 128 activation rows: handing a tile from role to role
//               takes some 600 cycles, more than the MMAs of 128 K take there: 37 x 14336 x 4096 17.0 us, with 128 19.5)
//   warp 1      eight MMAs per 128 K
//   warp 2      raw weights, a panel's 128 K (16 KB) a copy
//   8 or 16     epilogue: results from the accumulator, scaled
//   16 or 8     conversion: 32 codes a lane and tile of 64 K, ten instructions for eight
// Calls with few tiles are split over K; the slices' integer sums go to the
// workspace and a last launch adds and scales them (37 x 4096 x 14336: 20 us, whole 39).
//
// Bound by the weight stream and the hand-over for few rows (16 x 14336 x 4096 16 us, 3.6 TB/s), by the MMAs for many
// (1024 x 14336 x 4096 76 us, 1.58 PFLOP/s, the tensor pipe at 71 % of the kernel's cycles); both with the preparation.
//
// Waits are bounded, as in the 4-bit GEMM: one that gives up raises the error
// word, every other role ends, and what was issued is waited for.
#include "qmm_q8c.cuh"
#include "qmm_q4g_gemm.cuh"

namespace qmm {
namespace {

constexpr int kRaw = 8 * kQcSeg;      // bytes of a panel's 128 K
constexpr int kRestart = 8;           // times 128 K per accumulation where sums may pass 2^24
constexpr int kMaxBX = 256;
constexpr int kXMax = 8, kXMin = 4, kRawMax = 12;  // stages, at most: activations (and at least), raw weights
constexpr int kBars = (2 * kXMax + 2 * kQgStageMax + 2 * kRawMax + 4) * 8;  // bytes of the mbarriers
// Tiles of 128 K are for many activation rows: their MMAs take 1024 cycles, eight warps convert as fast,
// and 16 read the accumulator out while the MMAs wait for it (1024 x 14336 x 4096: 3.4 us of a unit's 21 with
// eight).  Tiles of 256 K are bound by the conversion.
__host__ __device__ constexpr int epi_warps(int kt) { return kt == 1 ? 16 : 8; }
constexpr int kTail = kBars + 32 + 4 * kMaxBX * 4;             // behind the rings: mbarriers, three words, the columns' factors
static_assert(kRawMax % 2 == 0 && kBars % 16 == 0, "rings of whole turns");

struct GemmParams {
    QcCall c;
    int* part;              // K slices: integer sums [ks][M][N]
    const float* xs;        // scales of the activation rows
    const uint32_t* xn;     // their sums of squares
    unsigned* err;
    int bx, nacc, accw, mtiles, ntiles, nraw, nx, nstage, ks;
    int ktiles;             // tiles in K
    int off_raw, off_bar;
    int wide;               // qc_wide_results
    int stall;
    unsigned stall_block;
};

struct Unit {
    int p0, n, nt;      // first activation row, their number, this block's row tile
    int split, j0, j1;  // K slice, its tiles
};

// KT: 128 K's in a tile
template <int CG, int KT>
__global__ void __launch_bounds__(kQgThreads, 1) q8c_gemm_kernel(const __grid_constant__ CUtensorMap tx, const GemmParams p) {
    extern __shared__ __align__(1024) uint8_t smraw[];
    uint8_t* sm = smraw + ((1024 - (smem_u32(smraw) & 1023)) & 1023);
    constexpr int kEpiWarps = epi_warps(KT), kEpiHalves = kEpiWarps / 4, kGroups = (24 - kEpiWarps) / 8, kConv0 = kQgEpi0 + kEpiWarps;
    constexpr int kWarpCols = kMaxBX / kEpiHalves;  // columns that an epilogue warp reads out, at most
    static_assert(kConv0 + 8 * kGroups == kQgThreads / 32, "every warp has a role");
    const QcCall& c = p.c;
    const QcWeights& w = c.w;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, M = c.a.M;
    uint64_t* bars = reinterpret_cast<uint64_t*>(sm + p.off_bar);
    uint64_t* x_full = bars;                       // activation tile landed (of a pair: both halves)
    uint64_t* x_empty = x_full + kXMax;          // and read by the MMAs (commit)
    uint64_t* full = x_empty + kXMax;            // converted weights in tensor memory
    uint64_t* empty = full + kQgStageMax;          // and read by the MMAs (commit)
    uint64_t* r_full = empty + kQgStageMax;        // raw weights landed
    uint64_t* r_empty = r_full + kRawMax;        // raw stage converted
    uint64_t* acc_full = r_empty + kRawMax;      // accumulator complete (commit)
    uint64_t* acc_empty = acc_full + 2;            // accumulator read
    uint32_t* tslot = reinterpret_cast<uint32_t*>(sm + p.off_bar + kBars);
    uint32_t* s_norm = tslot + 1;
    volatile int* flags = reinterpret_cast<volatile int*>(tslot + 2);
    float* s_xs = reinterpret_cast<float*>(tslot + 8);  // [epilogue warps][kWarpCols]
    const uint32_t rank = CG == 2 ? cluster_rank() : 0u;
    constexpr int kUnit = 16 * CG;  // the MMA's N is a multiple of 16, a pair's of 32
    const int first_unit = blockIdx.x / CG, unit_step = gridDim.x / CG;
    if (tid == 0) {
        for (int i = 0; i < kXMax; ++i) {
            mbar_init(smem_u32(&x_full[i]), 1);
            mbar_init(smem_u32(&x_empty[i]), 1);
        }
        for (int i = 0; i < kQgStageMax; ++i) {
            mbar_init(smem_u32(&full[i]), 8 * CG);
            mbar_init(smem_u32(&empty[i]), 1);
        }
        for (int i = 0; i < kRawMax; ++i) {
            mbar_init(smem_u32(&r_full[i]), 1);
            mbar_init(smem_u32(&r_empty[i]), 8);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(smem_u32(&acc_full[i]), 1);
            mbar_init(smem_u32(&acc_empty[i]), kEpiWarps * CG);
        }
        flags[0] = 0;
        *s_norm = 0u;
        fence_mbar_init();
    }
    if (warp == 1) {
        if (CG == 1) {
            asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(tslot)), "n"(kTcTmemCols)
                         : "memory");
            asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
        } else {
            asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(tslot)), "n"(kTcTmemCols)
                         : "memory");
            asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
        }
    }
    grid_dep_launch();
    tc_fence_before();
    __syncthreads();
    if (CG == 2) cluster_sync();  // the pair's barriers are initialised, its tensor memory is allocated
    tc_fence_after();
    const uint32_t tmem = *tslot;
    const int tiles_all = p.mtiles * p.ntiles, units = tiles_all * p.ks;
    // activation rows in tiles of one size, not full ones and a rest
    const int size = ((M + p.mtiles - 1) / p.mtiles + kUnit - 1) & ~(kUnit - 1);
    auto place = [&](int u) {
        Unit un;
        un.split = u / tiles_all;
        u -= un.split * tiles_all;
        const int st = u / p.ntiles;
        un.nt = (u - st * p.ntiles) * CG + (int)rank;
        un.p0 = st * size;
        un.n = max(min(size, M - un.p0), 0);
        un.j0 = (int)((long long)un.split * p.ktiles / p.ks);
        un.j1 = (int)((long long)(un.split + 1) * p.ktiles / p.ks);
        return un;
    };
    // an activation stage: 64-K pieces of the rows; of a pair, each block has half the rows
    const int half = p.bx / CG * 128;
    auto stage = [&](int s) { return sm + s * 2 * KT * half; };
    auto raw = [&](int s) { return sm + p.off_raw + s * KT * kRaw; };
    // 64-K pieces of tile j that hold any K
    auto halves = [&](int j) { return min(2 * KT, (w.K - j * 128 * KT + 63) / 64); };

    if (warp == 2) {
        // ------------------------------ raw weights: constant, so at once ------------------------------
        if (lane == 0) {
            QgRing r;
            bool ok = true, wrapped = false;
            int left = p.stall - 1;  // in 128 K
            for (int u = first_unit; u < units && ok; u += unit_step) {
                const Unit un = place(u);
                const int bytes = 8 * un.nt < w.RB ? qc_step(w, 8 * un.nt) : 0;
                const uint8_t* from = w.data + qc_row_block(w, 8 * un.nt);
                for (int j = un.j0; j < un.j1; ++j) {
                    // injected stall: this block's raw weights end here
                    if (p.stall && blockIdx.x == p.stall_block && (left -= KT) < 0) ok = false;
                    if (!ok || !(ok = qg_wait(smem_u32(&r_empty[r.s]), r.ph ^ 1u, flags, p.err))) break;
                    const uint32_t bar = smem_u32(&r_full[r.s]);
                    // a panel's segments of this K; row blocks, and K, past the last one keep what was there
                    const uint32_t all = (uint32_t)(bytes * min(KT, w.KS - j * KT));
                    mbar_arrive_tx(bar, all);
                    if (all > 0) bulk_g2s(smem_u32(raw(r.s)), from + (long long)j * KT * bytes, all, bar);
                    r.next(p.nraw);
                    wrapped |= r.s == 0;
                }
            }
            qg_drain(r, wrapped, p.nraw, r_full, flags, p.err);
        }
    } else if (warp == 0) {
        // ------------------------------ activations ------------------------------
        if (lane == 0) {
            asm volatile("prefetch.tensormap [%0];" ::"l"(&tx) : "memory");
            grid_dep_wait();
            QgRing g;
            bool ok = true, wrapped = false;
            for (int u = first_unit; u < units && ok; u += unit_step) {
                const Unit un = place(u);
                const int p0 = un.p0 + (int)rank * ((un.n + kUnit - 1) / kUnit * kUnit / CG);
                for (int j = un.j0; j < un.j1; ++j) {
                    if (!(ok = qg_wait(smem_u32(&x_empty[g.s]), g.ph ^ 1u, flags, p.err))) break;
                    uint32_t bar = smem_u32(&x_full[g.s]);
                    const uint32_t to = smem_u32(stage(g.s));
                    if (rank == 0) mbar_arrive_tx(bar, (uint32_t)(CG * 2 * KT * half));
                    if (CG == 2) bar = leader_addr(bar);
                    tma_4d<CG>(to, &tx, 0, p0, 0, 2 * KT * j, bar);
                    g.next(p.nx);
                    wrapped |= g.s == 0;
                }
            }
            // let every copy land before the block can exit (rank 0's barriers have both blocks')
            if (rank == 0) qg_drain(g, wrapped, p.nx, x_full, flags, p.err);
        }
    } else if (warp < kConv0) {
        // whether a sum may pass 2^24: the epilogue's and the MMAs' warps look for themselves
        grid_dep_wait();
        const uint32_t wnorm = __ldg(reinterpret_cast<const uint32_t*>(w.data + w.norm_off));
        uint32_t top = 0;
        for (int i = (warp == 1 ? 0 : warp - kQgEpi0 + 1) * 32 + lane; i < M; i += (kEpiWarps + 1) * 32) top = max(top, p.xn[i]);
        top = __reduce_max_sync(0xffffffffu, top);
        if (lane == 0) atomicMax(s_norm, top);
        asm volatile("bar.sync 1, %0;" ::"n"((kEpiWarps + 1) * 32) : "memory");
        const bool restart = (unsigned long long)*reinterpret_cast<volatile uint32_t*>(s_norm) * wnorm >= 1ull << 48;
        const int chunk = restart ? kRestart / KT : p.ktiles;
        if (warp == 1) {
            // ------------------------------ MMA issuer ------------------------------
            if (rank == 0) {
                // the whole warp runs the loop, so that its values are uniform, and one elected lane waits and issues
                const bool lead = elect_one();
                const uint64_t d0 = tc_sdesc128(smem_u32(stage(0)));
                const uint32_t lo0 = (uint32_t)d0, dhi = (uint32_t)(d0 >> 32);
                QgRing g, gx;
                int cc = 0, last = -1;  // accumulator uses; the last weight stage issued
                uint32_t last_ph = 0, ready = 0;  // the next stage's barrier, tested before this tile's MMAs are issued
                bool ok = true;
                for (int u = first_unit; u < units; u += unit_step) {
                    const Unit un = place(u);
                    const uint32_t idesc = tc_idesc((un.n + kUnit - 1) / kUnit * kUnit) + ((uint32_t)((CG - 1) * (kTcBW >> 4)) << 24);  // a pair: M = 256
                    for (int c0 = un.j0; c0 < un.j1; c0 += chunk, ++cc) {
                        const int ab = p.nacc == 2 ? (cc & 1) : 0, use = p.nacc == 2 ? (cc >> 1) : cc;
                        if (lead && ok && use > 0) ok = qg_wait(smem_u32(&acc_empty[ab]), (uint32_t)((use - 1) & 1), flags, p.err);
                        const uint32_t dt = tmem + (uint32_t)(ab * p.accw);
                        const int n = min(chunk, un.j1 - c0);
                        for (int i = 0; i < n; ++i) {
                            const int s = g.s;
                            const uint32_t ph = g.ph;
                            g.next(p.nstage);
                            const uint32_t next = mbar_test(smem_u32(&full[g.s]), g.ph);
                            if (lead && ok) ok = qg_wait(smem_u32(&x_full[gx.s]), gx.ph, flags, p.err) && (ready || qg_wait(smem_u32(&full[s]), ph, flags, p.err));
                            const int sx = gx.s;
                            gx.next(p.nx);
                            ready = next;
                            tc_fence_after();
                            const uint32_t x0 = lo0 + (uint32_t)((sx * 2 * KT * half) >> 4), a0 = tmem + (uint32_t)(p.nacc * p.accw + 64 * KT * s);
                            const int nh = halves(c0 + i);
                            __syncwarp();
                            if (lead && ok) {
#pragma unroll
                                for (int h = 0; h < 2 * KT; ++h) {
                                    if (h >= nh) break;
#pragma unroll
                                    for (int kk = 0; kk < 4; ++kk)
                                        qg_mma_tc<CG>(dt, a0 + 32 * h + 8 * kk, ((uint64_t)dhi << 32) | (x0 + (uint32_t)(h * half >> 4) + 2 * kk), idesc,
                                                      (i | h | kk) != 0 ? 1u : 0u);
                                }
                                qg_commit<CG>(smem_u32(&empty[s]));
                                qg_commit<CG>(smem_u32(&x_empty[sx]));
                                last = s;
                                last_ph = ph;
                            }
                        }
                        if (lead && ok) qg_commit<CG>(smem_u32(&acc_full[ab]));
                    }
                }
                // the last commits must land before tensor memory is released
                if (last >= 0) mbar_drain(smem_u32(&empty[last]), last_ph, flags, p.err);
            }
        } else {
            // ------------------------------ epilogue ------------------------------
            // chunks of 8 columns part, part + kEpiHalves, .. of the unit are this warp's
            const int ew = warp - kQgEpi0, q = warp & 3, part = ew >> 2;
            const uint32_t tq = (uint32_t)(32 * q) << 16;
            int cc = 0;
            bool ok = true;
            const float* sw = reinterpret_cast<const float*>(w.data + w.scale_off);
            // A unit's factors, asked for a unit ahead: this lane's row; the columns' go to shared memory, each
            // warp's own, in the order of its chunks.
            constexpr int kWords = kWarpCols / 32;
            float wn_next = 0.0f, bias_next = 0.0f, xs_next[kWords];
            float* table = s_xs + ew * kWarpCols;
            auto ask = [&](const Unit& un) {
                const int n = (8 * un.nt + 2 * q) * 16 + lane;
                wn_next = n < w.N ? __ldg(sw + n) : 0.0f;
                bias_next = c.bias && n < w.N ? c.bias[n] : 0.0f;
#pragma unroll
                for (int i = 0; i < kWords; ++i) {
                    const int m = kCols * (part + kEpiHalves * (4 * i + (lane >> 3))) + (lane & 7);
                    xs_next[i] = m < un.n ? p.xs[un.p0 + m] : 0.0f;
                }
            };
            if (first_unit < units) ask(place(first_unit));
            for (int u = first_unit; u < units && ok; u += unit_step) {
                const Unit un = place(u);
                const int nch = (un.n + kCols - 1) / kCols;
                const int n = (8 * un.nt + 2 * q) * 16 + lane;  // the tile's 128 rows are the lanes of the four quarters
                const bool on = n < w.N;
                const float wn = wn_next, bias = bias_next;
                __syncwarp();  // the last unit's have been read
#pragma unroll
                for (int i = 0; i < kWords; ++i) table[32 * i + lane] = xs_next[i];
                __syncwarp();
                if (u + unit_step < units) ask(place(u + unit_step));
                // 16-bit results go to memory four at a time where their place allows it, of four rows: a quad of lanes exchanges its 4 x 8 values
                // (a store a value and column took three times as long).  What a chunk needs is worked out before it:
                // this warp's chunks are kEpiHalves * kCols columns apart, and the kind of result is told apart outside of them.
                const bool wide = p.wide;
                const int sub = wide ? 2 * (lane & 3) : 0;  // the first of the columns that this lane writes
                const long long first = (long long)(un.p0 + kCols * part + sub) * w.N + n - (wide ? lane & 3 : 0) + (p.ks > 1 ? (long long)un.split * M * w.N : 0);
                const long long stride = (long long)kEpiHalves * kCols * w.N;
                const unsigned long long wn2 = f2pack(wn, wn);
                // Chunk i of this warp (its columns are `left` of eight), as `kind`.  whole: sums that a float may not hold.
                auto put = [&](auto kind, int i, int left, const float v[kCols], const int* whole) {
                    using Y = decltype(kind);
                    const long long o = first + i * stride;
                    if constexpr (std::is_same<Y, int>::value) {
                        int* to = p.part + o;
#pragma unroll
                        for (int e = 0; e < kCols; ++e, to += w.N)
                            if (on && e < left) *to = whole ? whole[e] : __float2int_rn(v[e]);
                    } else {
                        const float4 f0 = *reinterpret_cast<const float4*>(table + kCols * i), f1 = *reinterpret_cast<const float4*>(table + kCols * i + 4);
                        const float sx[kCols] = {f0.x, f0.y, f0.z, f0.w, f1.x, f1.y, f1.z, f1.w};
                        float y[kCols];
#pragma unroll
                        for (int e = 0; e < kCols; e += 2) {  // qc_scale, its products two at a time (a packed sum would be contracted with them)
                            const unsigned long long r = mul2(mul2(f2pack(v[e], v[e + 1]), wn2), f2pack(sx[e], sx[e + 1]));
                            y[e] = __fadd_rn(f2lo(r), bias);
                            y[e + 1] = __fadd_rn(f2hi(r), bias);
                        }
                        Y* to = static_cast<Y*>(c.y) + o;
                        if constexpr (std::is_same<Y, float>::value) {
#pragma unroll
                            for (int e = 0; e < kCols; ++e, to += w.N)
                                if (on && e < left) *to = y[e];
                        } else if (wide) {
                            uint32_t h[kCols / 2];  // columns 2 e, 2 e + 1
#pragma unroll
                            for (int e = 0; e < kCols / 2; ++e) {
                                if constexpr (std::is_same<Y, __half>::value) {
                                    const __half2 b = __floats2half2_rn(y[2 * e], y[2 * e + 1]);
                                    h[e] = *reinterpret_cast<const uint32_t*>(&b);
                                } else {
                                    const __nv_bfloat162 b = __floats2bfloat162_rn(y[2 * e], y[2 * e + 1]);
                                    h[e] = *reinterpret_cast<const uint32_t*>(&b);
                                }
                            }
                            const uint4 t = qg_quad_transpose(h[0], h[1], h[2], h[3], lane);  // columns sub, sub + 1 of the quad's rows
                            if (on && sub < left) *reinterpret_cast<uint2*>(to) = make_uint2(__byte_perm(t.x, t.y, 0x5410u), __byte_perm(t.z, t.w, 0x5410u));
                            if (on && sub + 1 < left) *reinterpret_cast<uint2*>(to + w.N) = make_uint2(__byte_perm(t.x, t.y, 0x7632u), __byte_perm(t.z, t.w, 0x7632u));
                        } else {
#pragma unroll
                            for (int e = 0; e < kCols; ++e, to += w.N)
                                if (on && e < left) *to = to_type<Y>(y[e]);
                        }
                    }
                };
                auto as_kind = [&](auto f) {
                    if (p.ks > 1) f(int());
                    else if (c.yt == X_F32) f(float());
                    else if (c.yt == X_F16) f(__half());
                    else f(__nv_bfloat16());
                };
                int sums[kWarpCols];  // local memory; restarted accumulations only
                for (int c0 = un.j0; c0 < un.j1; c0 += chunk, ++cc) {
                    const int ab = p.nacc == 2 ? (cc & 1) : 0, use = p.nacc == 2 ? (cc >> 1) : cc;
                    if (!(ok = qg_wait_warp(smem_u32(&acc_full[ab]), (uint32_t)(use & 1), false, flags, p.err))) break;
                    tc_fence_after();
                    __syncwarp();
                    const uint32_t acol = tmem + tq + (uint32_t)(ab * p.accw);
                    const bool begin = c0 == un.j0, end = c0 + chunk >= un.j1;
                    uint32_t r[kCols];
                    if (part < nch) tc_ld8(acol + kCols * part, r);
                    auto chunks = [&](auto take) {  // take(chunk of this warp, its columns, their sums)
#pragma unroll 1
                        for (int k = part, i = 0; k < nch; k += kEpiHalves, ++i) {
                            tc_wait_ld();
                            float v[kCols];
#pragma unroll
                            for (int e = 0; e < kCols; ++e) {
                                asm volatile("" : "+r"(r[e]));  // not used before the wait
                                v[e] = __uint_as_float(r[e]);
                            }
                            if (k + kEpiHalves < nch) tc_ld8(acol + kCols * (k + kEpiHalves), r);
                            take(i, un.n - kCols * k, v);
                        }
                    };
                    if (begin && end) {
                        as_kind([&](auto kind) { chunks([&](int i, int left, const float v[kCols]) { put(kind, i, left, v, nullptr); }); });
                    } else {
                        chunks([&](int i, int left, float v[kCols]) {
                            int* sum = sums + kCols * i;
#pragma unroll
                            for (int e = 0; e < kCols; ++e) {
                                sum[e] = (begin ? 0 : sum[e]) + __float2int_rn(v[e]);
                                v[e] = (float)sum[e];
                            }
                            if (end) as_kind([&](auto kind) { put(kind, i, left, v, sum); });
                        });
                    }
                    __syncwarp();
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) {
                        if (CG == 2) mbar_arrive_cluster(leader_addr(smem_u32(&acc_empty[ab])));
                        else mbar_arrive(smem_u32(&acc_empty[ab]));
                    }
                }
            }
        }
    } else {
        // ------------------------------ conversion ------------------------------
        const int cw = warp - kConv0, q = warp & 3, hh = (cw >> 2) & 1, grp = cw >> 3;  // row block 2 q + hh of a tile
        QgRing g, r;      // the next tile's weight and raw stage
        int turn = 0;     // the group that it is for
        uint32_t r_ready = 0;  // this group's next raw stage was seen to have landed
        int stored = -1;  // the stage of this warp's last tile, whose stores have not been waited for
        auto announce = [&]() {
            if (stored < 0) return;
            asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
            tc_fence_before();
            __syncwarp();
            if (lane == 0) {
                if (CG == 2) mbar_arrive_cluster(leader_addr(smem_u32(&full[stored])));
                else mbar_arrive(smem_u32(&full[stored]));
            }
            stored = -1;
        };
        // a 64-K tile's fragment registers: row g's in the even ones, row g + 8's in the odd ones
        auto convert = [&](const uint8_t* tile, uint32_t v[16]) {
            const uint4 a = reinterpret_cast<const uint4*>(tile)[lane], b = reinterpret_cast<const uint4*>(tile + 512)[lane];
            qc_half4(a.x, v[0], v[2]);
            qc_half4(b.x, v[1], v[3]);
            qc_half4(a.y, v[4], v[6]);
            qc_half4(b.y, v[5], v[7]);
            qc_half4(a.z, v[8], v[10]);
            qc_half4(b.z, v[9], v[11]);
            qc_half4(a.w, v[12], v[14]);
            qc_half4(b.w, v[13], v[15]);
        };
        bool ok = true;
        for (int u = first_unit; u < units && ok; u += unit_step) {
            const Unit un = place(u);
            const int step = 8 * un.nt < w.RB ? qc_step(w, 8 * un.nt) : 0;  // from 128 K to the next
            // The groups take tiles in turn, whatever a unit's number of them: a group that waits for
            // the release of tile t - nstage has waited for t - groups - nstage, so that with nstage >=
            // groups the stage's barrier is at most one phase behind the wait's parity.
            for (int j = un.j0; j < un.j1; ++j, turn = turn + 1 == kGroups ? 0 : turn + 1) {
                const QgRing at = g, ar = r;
                g.next(p.nstage);
                r.next(p.nraw);
                if (turn != grp) continue;
                if (!(ok = qg_wait_warp(smem_u32(&r_full[ar.s]), ar.ph, r_ready, flags, p.err))) break;
                // tested here, needed after the conversion
                const uint32_t e_ready = mbar_test(smem_u32(&empty[at.s]), at.ph ^ 1u);
                const uint8_t* seg = raw(ar.s) + (2 * q + hh) * kQcSeg;
                const uint32_t col = tmem + ((uint32_t)(32 * q + 16 * hh) << 16) + (uint32_t)(p.nacc * p.accw + 64 * KT * at.s);
                uint32_t v[16];
                convert(seg, v);
                announce();
                if (!(ok = qg_wait_warp(smem_u32(&empty[at.s]), at.ph ^ 1u, e_ready, flags, p.err))) break;
                QgRing rn = r;  // this group's next raw stage
                rn.skip(kGroups - 1, p.nraw);
                r_ready = mbar_test(smem_u32(&r_full[rn.s]), rn.ph);
                tc_fence_after();
                __syncwarp();
                tc_st_frag<16>(col, v);
#pragma unroll
                for (int h = 1; h < 2 * KT; ++h) {
                    convert(seg + (h >> 1) * step + 1024 * (h & 1), v);
                    if (h == 2 * KT - 1) {
                        __syncwarp();
                        if (lane == 0) mbar_arrive(smem_u32(&r_empty[ar.s]));
                    }
                    tc_st_frag<16>(col + 32 * h, v);
                }
                stored = at.s;
                if (p.nstage <= kGroups) announce();  // no stage to spare
            }
        }
        announce();
    }
    tc_fence_before();
    __syncthreads();
    if (CG == 2) {
        // After a wait that gave up, rank 1's last copies, which complete on rank 0's barriers, may be
        // ones that rank 0 never counted: both blocks stay for many times a copy's duration.
        if (flags[0]) {
            const long long t0 = clock64();
            while (clock64() - t0 < kQgQuiet) __nanosleep(1000);
            __syncwarp();
        }
        cluster_sync();  // neither block leaves while the other's MMAs, copies or arrivals may reach it
    }
    if (warp == 1) {
        tc_fence_after();
        if (CG == 1) asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "n"(kTcTmemCols) : "memory");
        else asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem), "n"(kTcTmemCols) : "memory");
    }
}

// y of the K slices' integer sums
__global__ void __launch_bounds__(256) q8c_sum_kernel(const int* part, int ks, int M, int N, const float* sw, const float* xs, const float* bias, void* y, int yt) {
    grid_dep_launch();
    grid_dep_wait();
    const int n = blockIdx.x * 256 + threadIdx.x, m = blockIdx.y;
    if (n >= N) return;
    const long long all = (long long)M * N, i = (long long)m * N + n;
    const float wn = __ldg(sw + n), sx = xs[m], b = bias ? bias[n] : 0.0f;  // on their way beside the sums
    int v = 0;
    for (int s0 = 0; s0 < ks; s0 += 4) {
        int u[4];
#pragma unroll
        for (int s = 0; s < 4; ++s) u[s] = s0 + s < ks ? __ldcg(part + (s0 + s) * all + i) : 0;
#pragma unroll
        for (int s = 0; s < 4; ++s) v += u[s];
    }
    x_store(y, yt, i, qc_scale((float)v, wn, sx, b));
}

template <int CG, int KT>
cudaError_t gemm_go(const QcGemmPlan& pl, const CUtensorMap& tx, const GemmParams& p, int smem_max, cudaStream_t s) {
    static unsigned long long done = 0;
    auto* k = q8c_gemm_kernel<CG, KT>;
    const cudaError_t e = ensure_smem(k, smem_max, done);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)pl.grid);
    cfg.blockDim = dim3(kQgThreads);
    cfg.dynamicSmemBytes = pl.smem;
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = CG;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = CG == 1 ? 1 : 2;
    return cudaLaunchKernelEx(&cfg, k, tx, p);
}

}  // namespace

QcGemmPlan plan_q8c_gemm(const QcCall& c, int sms, int smem_max) {
    QcGemmPlan pl;
    const QcWeights& w = c.w;
    const long long M = c.a.M;
    // Modelled cycles: a tile costs its MMAs (half a cycle a column, at least 40 each) or its conversion and
    // handing over (900; of 256 K 1100); a unit its prologue and, without a second accumulator, the epilogue that the
    // next unit's MMAs wait for; slices of K their sums' traffic and a launch.
    double best = 0;
    for (int cg = 1; cg <= 2; ++cg) {
        const int unit = 16 * cg, workers = sms / cg, most = cg == 2 ? kMaxBX : 128;
        const int ntiles = (w.RB + 8 * cg - 1) / (8 * cg);
        for (long long tiles = (M + most - 1) / most; tiles <= 8 + (M + most - 1) / most; ++tiles) {
            const int bx = (int)((M + tiles - 1) / tiles + unit - 1) / unit * unit;
            const long long mt = (M + bx - 1) / bx, un = (long long)ntiles * mt;
            const int kt = bx <= 128 ? 2 : 1, ktiles = (w.KS + kt - 1) / kt;
            const double mma = 8.0 * kt * (cg == 1 ? (bx < 40 ? 40.0 : (double)bx) : bx < 80 ? 40.0 : bx / 2.0), tile = mma > 700.0 + 200.0 * kt ? mma : 700.0 + 200.0 * kt;
            const double once = bx > 192 ? 1500.0 + 12.0 * bx : 1500.0;
            for (int ks = 1; ks <= ktiles && ks <= 16 && (ks == 1 || un * ks <= 2 * workers); ++ks) {
                const double waves = (double)((un * ks + workers - 1) / workers);
                const double cost = waves * ((double)((ktiles + ks - 1) / ks) * tile + once) + (ks > 1 ? 4000.0 + 8.0 * ks * M * w.N / 3000.0 : 0.0);
                if (best == 0 || cost < 0.98 * best) {
                    best = cost;
                    pl.cg = cg;
                    pl.kt = kt;
                    pl.bx = bx;
                    pl.ks = ks;
                    pl.mtiles = (int)mt;
                    pl.ntiles = ntiles;
                }
            }
            if (bx == unit) break;
        }
    }
    pl.accw = (pl.bx + 31) / 32 * 32;
    // With two accumulators the epilogue runs beside the next unit's MMAs (192 x 28672 x 4096 44 us, with one 47); where
    // there is no next unit their columns hold converted weights (192 x 14336 x 4096 25, with two 29).
    const long long units = (long long)pl.mtiles * pl.ntiles * pl.ks, workers = sms / pl.cg;
    pl.nacc = pl.bx <= 192 && units > workers ? 2 : 1;
    pl.nstage = (kTcTmemCols - pl.nacc * pl.accw) / (64 * pl.kt);
    if (pl.nstage > kQgStageMax) pl.nstage = kQgStageMax;
    const int stage = pl.bx / pl.cg * 256 * pl.kt, raw = kRaw * pl.kt, room = smem_max - kTail - 1024;
    // The raw ring is a multiple of the converting groups, so that whoever waits for a stage's next filling
    // has waited for its last one (copies may land out of order).  Activations come from L2: few stages;
    // the weights' trip to memory wants as many bytes on their way as there is room for.
    auto turns = [](int n, int most) { return (n < most ? n : most) / 2 * 2; };
    pl.nx = kXMin;
    while (pl.nx > 2 && pl.nx * stage + 4 * raw > room) --pl.nx;
    pl.nraw = turns((room - pl.nx * stage) / raw, kRawMax);
    pl.nx = (room - pl.nraw * raw) / stage < kXMax ? (room - pl.nraw * raw) / stage : kXMax;
    if (pl.nstage < 2 || pl.nx < 2 || pl.nraw < 2) return pl;
    pl.smem = (size_t)pl.nx * stage + (size_t)pl.nraw * raw + kTail + 1024;
    if (units > (1ll << 30)) return pl;
    pl.grid = (int)(units < workers ? units : workers) * pl.cg;
    auto r256 = [](size_t v) { return (v + 255) / 256 * 256; };
    pl.ws_scale = r256((size_t)M * w.KS * 256);
    pl.ws_norm = pl.ws_scale + r256((size_t)M * 4);
    pl.ws_part = pl.ws_norm + r256((size_t)M * 4);
    pl.workspace = pl.ws_part + (pl.ks > 1 ? (size_t)pl.ks * M * w.N * 4 : 0);
    pl.ok = true;
    return pl;
}

cudaError_t launch_q8c_gemm(const QcGemmPlan& pl, const QcCall& c, void* ws, unsigned* err, int stall, int smem_max, cudaStream_t s) {
    // single blocks have up to 128 activation rows, so tiles of 256 K; what no kernel is compiled for is refused
    auto* go = pl.cg == 2 && pl.kt == 2 ? gemm_go<2, 2> : pl.cg == 2 && pl.kt == 1 ? gemm_go<2, 1> : pl.cg == 1 && pl.kt == 2 ? gemm_go<1, 2> : nullptr;
    if (!go) return cudaErrorInvalidConfiguration;
    uint8_t* wsb = static_cast<uint8_t*>(ws);
    const int M = c.a.M;
    const long long pitch = (long long)c.w.KS * 128;
    float* xs = reinterpret_cast<float*>(wsb + pl.ws_scale);
    uint32_t* xn = reinterpret_cast<uint32_t*>(wsb + pl.ws_norm);
    cudaError_t e = launch_q8c_prep(c.a, c.w.K, QcPrep{wsb, xs, xn, pitch}, true, s);
    if (e != cudaSuccess) return e;
    // activations: 64 K x rows x 1 x pitch / 64; a box has a block's rows (half a pair's) and a tile's part of the last
    CUtensorMap tx;
    const unsigned long long xdims[4] = {64, (unsigned long long)M, 1, (unsigned long long)pitch / 64};
    const unsigned long long xstrides[3] = {(unsigned long long)pitch * 2, (unsigned long long)pitch * 2 * M, 128};
    const unsigned xbox[4] = {64, (unsigned)(pl.bx / pl.cg), 1, (unsigned)(2 * pl.kt)};
    if (!make_map_nd(&tx, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, wsb, 4, xdims, xstrides, xbox, CU_TENSOR_MAP_SWIZZLE_128B)) return cudaErrorInvalidValue;
    GemmParams p;
    p.c = c;
    p.part = reinterpret_cast<int*>(wsb + pl.ws_part);
    p.xs = xs;
    p.xn = xn;
    p.err = err;
    p.bx = pl.bx;
    p.nacc = pl.nacc;
    p.accw = pl.accw;
    p.mtiles = pl.mtiles;
    p.ntiles = pl.ntiles;
    p.nraw = pl.nraw;
    p.nx = pl.nx;
    p.nstage = pl.nstage;
    p.ks = pl.ks;
    p.wide = qc_wide_results(c, pl.ks);
    p.stall = stall;
    p.stall_block = (unsigned)pl.cg - 1u;  // of a pair the second one, whose partner finds out by its own waits
    p.ktiles = (c.w.KS + pl.kt - 1) / pl.kt;
    p.off_raw = pl.nx * (pl.bx / pl.cg) * 256 * pl.kt;
    p.off_bar = p.off_raw + pl.nraw * kRaw * pl.kt;
    e = go(pl, tx, p, smem_max, s);
    if (e != cudaSuccess || pl.ks == 1) return e;
    const dim3 grid((unsigned)((c.w.N + 255) / 256), (unsigned)M);
    return launch_pdl_2d(q8c_sum_kernel, grid.x, grid.y, 256, 0, s, (const int*)p.part, pl.ks, M, c.w.N, reinterpret_cast<const float*>(c.w.data + c.w.scale_off),
                         (const float*)xs, c.bias, c.y, c.yt);
}

}  // namespace qmm
