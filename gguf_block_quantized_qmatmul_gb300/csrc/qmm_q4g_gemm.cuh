// qmm_q4g_gemm.cuh -- products of 4-bit group-scale weights with many
// activation rows on tcgen05: prompts through a dense linear, and the
// experts' products of a batch (grouped by expert, any number of rows each).
//
// Mathematics.  Weight rows and activation rows are brought into f16's range
// by a power of two each (the weights' at layout time, the activations' by the
// preparation launch; f16 activations keep theirs), and
//   y = 2^-(a + b) sum_k f16(s 2^a (q - z)) (x 2^b).
// s 2^a and q - z are exact in f16, their product is rounded to 11 bits.  It is
// exact where |q - z| is 0 or a power of two (half of the codes with a zero
// point of 8, five of sixteen with one of 0 or 15), and with a bf16 scale up to
// 8 and at the even ones.  So the sum's error is below that of rounding an f16
// result (with it 1.33 times the error of that rounding alone, measured with
// zero points of 6 to 9 and f16 scales), and far below a bf16 one.  f16 gate
// and up products would multiply two such sums (1.6 times), so they take the
// weights' rests as well, v = hi + lo, which makes s (q - z), of at most 16
// significant bits, exact.  bf16 activations are exact in f16 after scaling
// (values under 2^-29 of their row's largest lose bits).  f32 activations are
// two pieces too, 22 bits, and three MMAs: hi lo + lo hi + hi hi.
//
// One persistent block per SM over units: 128 weight rows (8 row blocks, the
// MMA's M) x up to bx activation rows of one expert (its N, rounded up to 16).
// With one piece, two blocks work as a pair (cta_group::2) on 256 weight rows:
// each converts its own 128, holds half of the activation rows and reads out its
// own accumulator rows; rank 0's MMA thread works for both.  A block alone has to
// write and read every activation row of its tile in its shared memory for 128
// weight rows, 128 bytes a cycle at the MMAs' peak, all that there is.
//   warp 0      one thread: activation tiles (128 K, two halves with 128-byte
//               swizzle), one 4-D box each (several made this thread's issue the
//               limit, 850 cycles a tile); the experts' rows were put in sorted
//               order by the preparation launch (gathering four rows a copy here
//               took 90 cycles a copy)
//   warp 1      one elected lane: eight MMAs a pass per tile of 128 K, A in tensor
//               memory, B in shared memory.  (With tiles of 64 K its wait, commits and
//               bookkeeping, about 300 cycles a tile alone and 500 beside the other
//               warps, held the MMAs up.)
//   warp 2      one thread: raw weights, a 2-D box of eight row blocks per segment
//               (a copy per row block took 300 cycles)
//   warps 3-10  epilogue: accumulator columns to registers, scaled; the experts'
//               first product takes its up row from the lane eight away (paired
//               layout) for silu(g) u
//   warps 11-26 conversion: a lane's uint4 of codes becomes fragment registers
//               and goes to tensor memory as they are (16-lane x 128-bit
//               stores); two groups of eight warps, a row block each, every other
//               tile
// The weights are bound for tensor memory, so shared memory feeds only the
// activation tiles to the MMAs.  The tensor core's f32 sums truncate, which f32
// results would show: the small products (hi lo, lo hi) of a tile go first,
// while the accumulator is small, the accumulator is restarted every kQgChunk
// tiles, and the epilogue adds the chunks in registers (error of 37 x 14336 x
// 4096: 9.8e-7 with the three passes in turn and two tiles a chunk, 6.6e-7 with
// the small ones first, 2.2e-7 with one tile as well, for 1.5 us more; the call
// takes 33.7).  The chunks' sums do not fit the epilogue's 72 registers: f32
// calls keep 216 bytes a thread in local memory.  A dense call with fewer units than SMs is split over K as well, and a
// last launch adds the slices.
//
// Measured, in a graph: 1024 x 14336 x 4096 f16 75 us (1.60 PFLOP/s; the tensor
// pipe 65 % of all cycles, the MMAs are the bound and the rest is three units a
// pair that do not overlap their last epilogue); 2048 tokens x 8 of 64 experts,
// 2048 -> 2 x 1024 bf16 139 us with its preparation (12 us), 1024 -> 2048 f16 125
// us with preparation (12) and combination (25).  There 256 rows an expert do
// not repay one conversion of its weights: two thirds of the issue slots are
// taken, and four converting warps and two epilogue warps a scheduler share them.
//
// Waits are bounded.  One that gives up raises the error word and the block's
// abort flag, its warp leaves its role, every other wait of the block ends with
// the flag and the other block's by its own limit; copies and MMAs that were
// issued are waited for before shared and tensor memory are given back.
#pragma once

#include <type_traits>

#include "qmm_q4g_rows.cuh"

namespace qmm {

constexpr int kQgEpiWarps = 8, kQgConvWarps = 16;
constexpr int kQgEpiHalves = kQgEpiWarps / 4;   // epilogue warps per TMEM lane quarter
constexpr int kQgGroups = kQgConvWarps / 8;     // converting groups: a warp per row block of a tile
constexpr int kQgEpi0 = 3, kQgConv0 = kQgEpi0 + kQgEpiWarps;
constexpr int kQgThreads = (kQgConv0 + kQgConvWarps) * 32;
constexpr int kQgBX1 = 256, kQgBXA = 128, kQgBX2 = 64;  // activation rows per tile, at most: one piece, two of the weights, two of both
constexpr int kQgRawMax = 6, kQgXMax = 8, kQgStageMax = 8;  // stages, at most: raw weights, activations, converted weights
constexpr int kQgChunk = 1;      // tiles per accumulation chunk (two pieces of the activations)
constexpr int kCols = 8;         // accumulator columns that an epilogue warp takes at a time (with 16, 170 bytes a thread were spilled)
constexpr int kQgMaxE = 512;     // experts of a grouped call
constexpr long long kQgQuiet = 1ll << 16;  // clocks (some 35 us) that a pair stays after a wait that gave up
constexpr int kQgTab = 64;       // units of a block that are looked up at its start; later ones when they are taken

struct QgGemmParams {
    QgCall c;
    float* part;          // P_DOWN: [T top_k][N]
    const float* xs;      // 2^-b per activation row (experts: per sorted position); NULL: 1
    const float* wis;     // 2^-a per weight row, layout order
    unsigned* err;
    int bx, nacc, accw, mtiles, ntiles, nraw, nx, nstage;
    int ks;               // K slices (dense): f32 partial outputs [ks][M][N]
    int off_raw, off_bar;
    int stall;             // test hook: block stall_block copies only stall - 1 tiles of its raw weights; 0: all
    unsigned stall_block;
};

// 2 R columns of 16 lanes from R fragment registers: lane 4 g + t's registers 2 j, 2 j + 1 are column 4 j + t of lanes g, g + 8
template <int R>
__device__ __forceinline__ void tc_st_frag(uint32_t taddr, const uint32_t* v) {
    static_assert(R == 16 || R == 8, "one or two pieces");
    if constexpr (R == 16)
        asm volatile(
            "tcgen05.st.sync.aligned.16x128b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(taddr),
            "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(v[8]), "r"(v[9]),
            "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15])
            : "memory");
    else
        asm volatile("tcgen05.st.sync.aligned.16x128b.x4.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(taddr), "r"(v[0]), "r"(v[1]),
                     "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
                     : "memory");
}

// Pairs of blocks (cta_group::2): a cluster of two, whose rank 0 issues the MMAs of both.
__device__ __forceinline__ uint32_t cluster_rank() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
    asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// the address, in the cluster's shared memory, of rank 0's copy of a shared variable
__device__ __forceinline__ uint32_t leader_addr(uint32_t a) {
    uint32_t r;
    asm("mapa.shared::cluster.u32 %0, %1, 0;" : "=r"(r) : "r"(a));
    return r;
}
// What these arrivals announce is tensor memory (ordered by the tcgen05 fences before them and
// after the wait); with cluster-scope release and acquire a tile took 990 cycles, not 670.
__device__ __forceinline__ void mbar_arrive_cluster(uint32_t a) {
    asm volatile("mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" ::"r"(a) : "memory");
}
// One TMA box of a 4-D tensor map; CG = 2: completing on a barrier of the pair's leader.
template <int CG>
__device__ __forceinline__ void tma_4d(uint32_t dst, const CUtensorMap* map, int x, int y, int z, int t, uint32_t bar) {
    if (CG == 1)
        asm volatile(
            "cp.async.bulk.tensor.4d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(dst),
            "l"(map), "r"(x), "r"(y), "r"(z), "r"(t), "r"(bar)
            : "memory");
    else
        asm volatile(
            "cp.async.bulk.tensor.4d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(
                dst),
            "l"(map), "r"(x), "r"(y), "r"(z), "r"(t), "r"(bar)
            : "memory");
}
template <int CG>
__device__ __forceinline__ void qg_mma_tc(uint32_t tmem, uint32_t ta, uint64_t db, uint32_t idesc, uint32_t accumulate) {
    if (CG == 1)
        tc_mma(tmem, ta, db, idesc, accumulate);
    else
        asm volatile(
            "{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %4, 0;\n\t"
            "tcgen05.mma.cta_group::2.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(tmem),
            "r"(ta), "l"(db), "r"(idesc), "r"(accumulate)
            : "memory");
}
// A weight row's power of two (2^-120 to 2^118) in two factors: one of 2^-60 to 2^60, and the rest.
// A sum (of up to 2^51) is multiplied by the one, its activation row's power of two and, where some
// row of the warp's has one, the rest: no step leaves the f32 range where the result does not.
// (The two powers' product leaves it for results below 2e-35, and made 0 times infinity of a sum of 0.
// With a multiplication by the rest for every sum gate_up of 2048 tokens took 155.6 us, not 142.)
struct QgFactor {
    float near, rest;
};
__device__ __forceinline__ QgFactor qg_factor(float pow2) {
    const int e = max((int)(__float_as_uint(pow2) >> 23) - 127, -120), n = max(min(e, 60), -60);  // 0: no row
    return {__uint_as_float((uint32_t)(127 + n) << 23), __uint_as_float((uint32_t)(127 + e - n) << 23)};
}

// the completion of the MMAs before it arrives on this barrier, in both blocks of a pair
template <int CG>
__device__ __forceinline__ void qg_commit(uint32_t bar) {
    if (CG == 1)
        tc_commit(bar);
    else
        asm volatile("tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(bar),
                     "h"((uint16_t)3)
                     : "memory");
}

__device__ __forceinline__ void tc_ld8(uint32_t taddr, uint32_t r[8]) {
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
                 : "r"(taddr));
}

// true in one lane of a converged warp
__device__ __forceinline__ bool elect_one() {
    uint32_t p;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(p));
    return p != 0;
}

// Words s0 .. s0 + WORDS - 1 of a lane's four of 64-K tile h of a segment: fragment registers of
// their f16 weights (and their rests).  g: the group's constants (with one group a segment, those
// of tile 0 serve tile 1).
struct QgGroup {
    uint32_t zl, zh;
    __half2 s0, s1;
};
template <int PA, int NG, int WORDS>
__device__ __forceinline__ void qg_convert(const uint8_t* seg, const uint4& q, int h, int s0, int lane, uint32_t magic, float m0, float m1, QgGroup& g, uint32_t* hi,
                                           uint32_t* lo) {
    const uint32_t word[4] = {q.x, q.y, q.z, q.w};
    const uint32_t* sw = reinterpret_cast<const uint32_t*>(seg + 2 * kQgTile + (lane >> 2) * (8 * NG));
#pragma unroll
    for (int s = s0; s < s0 + WORDS; ++s) {
        if ((s == 0 && (NG != 1 || h == 0)) || (NG == 4 && s == 2)) {
            const int gi = NG == 1 ? 0 : NG == 2 ? h : 2 * h + (s >> 1);
            const uint2 v = *reinterpret_cast<const uint2*>(sw + 2 * gi);
            g.zl = qg_zero<false>(v.x, false);
            g.zh = qg_zero<false>(v.y, true);
            g.s0 = __float2half2_rn(qg_scale(v.x) * m0);
            g.s1 = __float2half2_rn(qg_scale(v.y) * m1);
        }
        uint32_t a[4];
        qg_codes<false>(word[s], magic, g.zl, g.zh, a);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const __half2 c = *reinterpret_cast<__half2*>(&a[i]);
            const __half2 sc = i & 1 ? g.s1 : g.s0;
            const __half2 p = __hmul2(c, sc);
            hi[4 * (s - s0) + i] = *reinterpret_cast<const uint32_t*>(&p);
            if (PA == 2) {
                const __half2 r = __hfma2(c, sc, __hneg2(p));
                lo[4 * (s - s0) + i] = *reinterpret_cast<const uint32_t*>(&r);
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
    int e, p0, n, nt;  // expert, first position (row of x in a dense call), activation rows, this block's row tile
    int split, j0, j1; // K slice, its tiles (segments of 128 K)
};

// PA pieces of the weights, PX of the activations
template <int PA, int PX, int NG, int CG>
__global__ void __launch_bounds__(kQgThreads, 1) q4g_gemm_kernel(const __grid_constant__ CUtensorMap tx, const __grid_constant__ CUtensorMap tw, const QgGemmParams p) {
    extern __shared__ __align__(1024) uint8_t smraw[];
    uint8_t* sm = smraw + ((1024 - (smem_u32(smraw) & 1023)) & 1023);
    const QgCall& c = p.c;
    const QgWeights& w = c.w;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    uint64_t* bars = reinterpret_cast<uint64_t*>(sm + p.off_bar);
    uint64_t* x_full = bars;                       // activation tile landed (of a pair: both halves)
    uint64_t* x_empty = x_full + kQgXMax;          // and read by the MMAs (commit)
    uint64_t* full = x_empty + kQgXMax;            // converted weights in tensor memory
    uint64_t* empty = full + kQgStageMax;          // and read by the MMAs (commit)
    uint64_t* r_full = empty + kQgStageMax;        // raw weights landed
    uint64_t* r_empty = r_full + kQgRawMax;        // raw stage converted
    uint64_t* acc_full = r_empty + kQgRawMax;      // accumulator complete (commit)
    uint64_t* acc_empty = acc_full + 2;            // accumulator read
    static_assert(kQgXMax % kQgGroups == 0 && kQgRawMax % kQgGroups == 0, "rings of whole turns");
    uint64_t* tab_full = acc_empty + 2;            // a unit's column tables, of the epilogue
    static_assert((2 * kQgXMax + 2 * kQgStageMax + 2 * kQgRawMax + 6) * 8 <= 448, "mbarriers overlap the TMEM slot");
    uint32_t* tslot = reinterpret_cast<uint32_t*>(sm + p.off_bar + 448);
    volatile int* flags = reinterpret_cast<volatile int*>(sm + p.off_bar + 480);
    int* col_slot = reinterpret_cast<int*>(sm + p.off_bar + 512);             // [2][kQgBX1]
    float* col_scale = reinterpret_cast<float*>(col_slot + 2 * kQgBX1);       // [2][kQgBX1]
    int4* tab = reinterpret_cast<int4*>(col_scale + 2 * kQgBX1);                 // [kQgTab] this block's units: expert and slice, p0, n, nt
    int* ts = reinterpret_cast<int*>(tab + kQgTab);                           // [E + 1] activation tiles before each expert
    int* po = ts + w.E + 1;                                                   // [E + 1] activation rows before each expert
    const uint32_t rank = CG == 2 ? cluster_rank() : 0u;
    constexpr int kUnit = 16 * CG;  // the MMA's N is a multiple of 16, a pair's of 32
    const int first_unit = blockIdx.x / CG, unit_step = gridDim.x / CG;
    const bool grouped = c.op != P_DENSE;
    const int slots = grouped ? c.r.T * c.r.top_k : c.M;
    if (tid == 0) {
        for (int i = 0; i < kQgXMax; ++i) {
            mbar_init(smem_u32(&x_full[i]), 1);
            mbar_init(smem_u32(&x_empty[i]), 1);
        }
        for (int i = 0; i < kQgStageMax; ++i) {
            mbar_init(smem_u32(&full[i]), 8 * CG);
            mbar_init(smem_u32(&empty[i]), 1);
        }
        for (int i = 0; i < kQgRawMax; ++i) {
            mbar_init(smem_u32(&r_full[i]), 1);
            mbar_init(smem_u32(&r_empty[i]), 8);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(smem_u32(&acc_full[i]), 1);
            mbar_init(smem_u32(&acc_empty[i]), kQgEpiWarps * CG);
            mbar_init(smem_u32(&tab_full[i]), kQgEpiWarps);
        }
        flags[0] = 0;
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
    if (grouped) grid_dep_wait();
    if (warp == 0) {
        if (grouped) {
            for (int e = lane; e <= w.E; e += 32) po[e] = min(max(__ldg(c.r.offsets + e), 0), slots);
            __syncwarp();
            const int per = (w.E + 31) / 32;
            int mine = 0;
            for (int i = 0; i < per; ++i) {
                const int e = lane * per + i;
                if (e < w.E) mine += (max(po[e + 1] - po[e], 0) + p.bx - 1) / p.bx;
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
                pre += (max(po[e + 1] - po[e], 0) + p.bx - 1) / p.bx;
            }
        } else if (lane == 0) {
            ts[0] = 0;
            ts[1] = p.mtiles;
            po[0] = 0;
            po[1] = c.M;
        }
    }
    tc_fence_before();
    __syncthreads();
    if (CG == 2) cluster_sync();  // the pair's barriers are initialised, its tensor memory is allocated
    tc_fence_after();
    const uint32_t tmem = *tslot;
    const int tiles_all = ts[w.E] * p.ntiles, units = tiles_all * p.ks;
    auto find = [&](int u) {
        QgUnit un;
        un.split = u / tiles_all;
        u -= un.split * tiles_all;
        const int st = u / p.ntiles;
        un.nt = (u - st * p.ntiles) * CG + (int)rank;
        int lo = 0, hi = w.E;  // ts[lo] <= st < ts[hi]
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (ts[mid] <= st) lo = mid;
            else hi = mid;
        }
        un.e = lo;
        const int first = po[lo], end = po[lo + 1];
        // an expert's rows in tiles of one size, not full ones and a rest
        const int tiles = ts[lo + 1] - ts[lo];
        const int size = ((end - first + tiles - 1) / tiles + kUnit - 1) & ~(kUnit - 1);
        un.p0 = first + (st - ts[lo]) * size;
        un.n = min(size, end - un.p0);
        return un;
    };
    // Looked up once, not by each of the warps that take the unit: that was a tenth of all instructions
    // and 1500 cycles at each unit's start.
    for (int i = tid; i < kQgTab && first_unit + i * unit_step < units; i += kQgThreads) {
        const QgUnit un = find(first_unit + i * unit_step);
        tab[i] = make_int4(un.e | un.split << 16, un.p0, un.n, un.nt);
    }
    __syncthreads();
    auto place = [&](int u, int i) {  // u: the block's unit i
        QgUnit un;
        if (i < kQgTab) {
            const int4 v = tab[i];
            un.e = v.x & 0xffff;
            un.split = v.x >> 16;
            un.p0 = v.y;
            un.n = v.z;
            un.nt = v.w;
        } else {
            un = find(u);
        }
        un.j0 = 0;
        un.j1 = w.KS;
        if (p.ks > 1) {
            un.j0 = un.split * w.KS / p.ks;
            un.j1 = (un.split + 1) * w.KS / p.ks;
        }
        return un;
    };
    if (!grouped && warp != 2) grid_dep_wait();  // weights are constant: their copies may start at once
    // an activation stage: two 64-K halves of the rows' pieces; of a pair, each block has half the rows
    const int half = p.bx / CG * 128;
    auto stage = [&](int s) { return sm + s * 2 * PX * half; };
    const int seg_bytes = qg_seg_bytes(NG);
    auto raw = [&](int s) { return sm + p.off_raw + s * 8 * seg_bytes; };
    // 64-K halves of tile j that hold any K
    auto halves = [&](int j) { return w.K - j * kQgSegK > 64 ? 2 : 1; };

    if (warp == 0) {
        // ------------------------------ activations ------------------------------
        if (lane == 0) {
            QgRing g;
            bool ok = true, wrapped = false;
            for (int u = first_unit, ui = 0; u < units && ok; u += unit_step, ++ui) {
                const QgUnit un = place(u, ui);
                const int p0 = un.p0 + (int)rank * ((un.n + kUnit - 1) / kUnit * kUnit / CG);
                for (int j = un.j0; j < un.j1; ++j) {
                    if (!(ok = qg_wait(smem_u32(&x_empty[g.s]), g.ph ^ 1u, flags, p.err))) break;
                    uint32_t bar = smem_u32(&x_full[g.s]);
                    const uint32_t to = smem_u32(stage(g.s));
                    if (rank == 0) mbar_arrive_tx(bar, (uint32_t)(CG * PX * 2 * half));
                    if (CG == 2) bar = leader_addr(bar);
                    tma_4d<CG>(to, &tx, 0, p0, 0, 2 * j, bar);
                    g.next(p.nx);
                    wrapped |= g.s == 0;
                }
            }
            // let every copy land before the block can exit (rank 0's barriers have both blocks')
            if (rank == 0) qg_drain(g, wrapped, p.nx, x_full, flags, p.err);
        }
    } else if (warp == 1) {
        // ------------------------------ MMA issuer ------------------------------
        if (rank == 0) {
            // The whole warp runs the loop, so that its values are uniform, and one elected lane
            // issues: inside a one-lane branch every MMA's operands take detours to uniform
            // registers (58 cycles an MMA and 410 a tile, against 128 cycles of MMAs at 64 rows).
            // That lane alone waits: after a wait that gave up it goes through the loop with the
            // others and does nothing more.  (Votes on its waits: 37 x 14336 x 4096 f32 34.2 us, not 33.1.)
            const bool lead = elect_one();
            const uint64_t d0 = tc_sdesc128(smem_u32(stage(0)));
            const uint32_t lo0 = (uint32_t)d0, dhi = (uint32_t)(d0 >> 32);
            QgRing g;
            QgRing gx;              // activation stage
            int cc = 0, last = -1;  // accumulator uses; the last weight stage issued
            uint32_t last_ph = 0;
            bool ok = true;
            uint32_t ready = 0;  // the next stage's barrier, tested before this tile's MMAs are issued
            for (int u = first_unit, ui = 0; u < units; u += unit_step, ++ui) {
                const QgUnit un = place(u, ui);
                const uint32_t idesc = tc_idesc((un.n + kUnit - 1) / kUnit * kUnit) + ((uint32_t)((CG - 1) * (kTcBW >> 4)) << 24);  // a pair: M = 256
                const int chunk = PX == 2 ? kQgChunk : w.KS;
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
                        const uint32_t x0 = lo0 + (uint32_t)((sx * 2 * PX * half) >> 4), a0 = tmem + (uint32_t)(p.nacc * p.accw + 64 * PA * s);
                        const int nh = halves(c0 + i);
                        __syncwarp();
                        if (lead && ok) {
                            // the small products first, while the accumulator is small: adding to it truncates
                            constexpr int kPasses = PA + PX - 1;  // weights, activations: hi lo, lo hi, hi hi (one piece: hi)
#pragma unroll
                            for (int pass = 0; pass < kPasses; ++pass) {
                                const bool wlo = PA == 2 && pass == kPasses - 2, xlo = PX == 2 && pass == 0;
#pragma unroll
                                for (int h = 0; h < 2; ++h) {
                                    if (h == 1 && nh == 1) break;
                                    const uint32_t wa = a0 + 32 * h + (wlo ? 64 : 0), xb = x0 + (uint32_t)((h * PX + (xlo ? 1 : 0)) * half >> 4);
#pragma unroll
                                    for (int kk = 0; kk < 4; ++kk)
                                        qg_mma_tc<CG>(dt, wa + 8 * kk, ((uint64_t)dhi << 32) | (xb + 2 * kk), idesc, (i | h | pass | kk) != 0 ? 1u : 0u);
                                }
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
    } else if (warp == 2) {
        // ------------------------------ raw weights ------------------------------
        if (lane == 0) {
            QgRing r;
            bool ok = true, wrapped = false;
            int left = p.stall - 1;
            for (int u = first_unit, ui = 0; u < units && ok; u += unit_step, ++ui) {
                const QgUnit un = place(u, ui);
                for (int j = un.j0; j < un.j1; ++j) {
                    // injected stall: this block's raw weights end here
                    if (p.stall && blockIdx.x == p.stall_block && --left < 0) ok = false;
                    if (!ok || !(ok = qg_wait(smem_u32(&r_empty[r.s]), r.ph ^ 1u, flags, p.err))) break;
                    const uint32_t bar = smem_u32(&r_full[r.s]);
                    mbar_arrive_tx(bar, (uint32_t)(8 * seg_bytes));
                    tma_2d(smem_u32(raw(r.s)), &tw, j * (seg_bytes / 8), un.e * w.RB + 8 * un.nt, bar);
                    r.next(p.nraw);
                    wrapped |= r.s == 0;
                }
            }
            qg_drain(r, wrapped, p.nraw, r_full, flags, p.err);
        }
    } else if (warp < kQgConv0) {
        // ------------------------------ epilogue ------------------------------
        const int ew = warp - kQgEpi0, q = warp & 3, half = ew >> 2;  // column chunks half, half + kQgEpiHalves, ...
        const uint32_t tq = (uint32_t)(32 * q) << 16;
        int cc = 0;
        bool ok = true;
        const int chunk = PX == 2 ? kQgChunk : w.KS;
        const int F = w.N / 2;
        // A unit's column tables (slot or row, factor): a thread a column, copied a unit ahead (loaded
        // at the unit's start they took 4000 cycles of some 17000).  And the factor of this lane's row.
        static_assert(kQgEpiWarps * 32 >= kQgBX1, "a thread per column");
        float wsn_next = 0.0f;
        auto ask = [&](const QgUnit& un, int b) {
            const int col = ew * 32 + lane;
            int* ds = col_slot + b * kQgBX1 + col;
            float* dc = col_scale + b * kQgBX1 + col;
            const bool on = col < un.n;
            if (on && grouped) cp_async4(smem_u32(ds), c.r.order + un.p0 + col);
            else *ds = on ? un.p0 + col : -1;
            if (on && p.xs) cp_async4(smem_u32(dc), p.xs + un.p0 + col);
            else *dc = 1.0f;
            cp_async_commit();
            const int rb = 8 * un.nt + 2 * q + (lane >> 4);
            wsn_next = rb < w.RB ? __ldg(p.wis + ((long long)un.e * w.RB + rb) * 16 + (lane & 15)) : 0.0f;
        };
        QgUnit un_next = {};
        if (first_unit < units) {
            un_next = place(first_unit, 0);
            ask(un_next, 0);
        }
        for (int u = first_unit, ui = 0; u < units && ok; u += unit_step, ++ui) {
            const QgUnit un = un_next;
            const float wsn = wsn_next;
            const int nch = (un.n + kCols - 1) / kCols;
            const int rb = 8 * un.nt + 2 * q + (lane >> 4);
            const int n = rb < w.RB ? qg_row(w, rb, lane & 15) : -1;
            const int* my_slot = col_slot + (ui & 1) * kQgBX1;
            const float* my_scale = col_scale + (ui & 1) * kQgBX1;
            // This warp's part of the tables has landed, and it no longer reads the last unit's; once all
            // have, the next unit's may be asked for.
            cp_async_wait<0>();
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_u32(&tab_full[ui & 1]));
            if (!(ok = qg_wait_warp(smem_u32(&tab_full[ui & 1]), (uint32_t)(ui >> 1) & 1u, false, flags, p.err))) break;
            __syncwarp();
            if (u + unit_step < units) {
                un_next = place(u + unit_step, ui + 1);
                ask(un_next, (ui + 1) & 1);
            }
            const float wup = __shfl_xor_sync(0xffffffffu, wsn, 8);  // the paired row's factor
            const bool up = (lane & 8) != 0;  // of a pair of rows: lanes r < 8 have gate rows, r + 8 their up rows
            const QgFactor wn = qg_factor(wsn), wg = qg_factor(up ? wup : wsn), wu = qg_factor(up ? wsn : wup);
            const bool rest = __any_sync(0xffffffffu, wg.rest != 1.0f || wu.rest != 1.0f);
            auto put_as = [&](auto* y, int k, const float v[kCols]) {  // columns kCols k..
                using Y = typename std::remove_pointer<decltype(y)>::type;
                if (c.op == P_GATE_UP) {
                    // the lane with the gate row finishes columns 0..3, the one with the up row 4..7
                    const int f = rb * 8 + (lane & 7);
                    const bool on = rb < w.RB && f < F;
                    const uint32_t row = (uint32_t)F * (uint32_t)sizeof(Y);
                    char* base = reinterpret_cast<char*>(y + f);
                    const int4 s4 = *reinterpret_cast<const int4*>(my_slot + kCols * k + (up ? 4 : 0));
                    const float4 x4 = *reinterpret_cast<const float4*>(my_scale + kCols * k + (up ? 4 : 0));
                    const int sl[4] = {s4.x, s4.y, s4.z, s4.w};
                    const float xc[4] = {x4.x, x4.y, x4.z, x4.w};
                    float gt[4], ut[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const float got = __shfl_xor_sync(0xffffffffu, up ? v[i] : v[i + 4], 8), mine = up ? v[i + 4] : v[i];
                        gt[i] = (up ? got : mine) * wg.near * xc[i];
                        ut[i] = (up ? mine : got) * wu.near * xc[i];
                    }
                    if (rest) {
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            gt[i] *= wg.rest;
                            ut[i] *= wu.rest;
                        }
                    }
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const float r = PX == 2 ? swiglu(gt[i], ut[i]) : swiglu_fast(gt[i], ut[i]);
                        if (on && (unsigned)sl[i] < (unsigned)slots) *reinterpret_cast<Y*>(base + (uint64_t)(uint32_t)sl[i] * row) = to_type<Y>(r);
                    }
                } else if (n >= 0) {
                    const uint32_t row = (uint32_t)w.N * (uint32_t)sizeof(Y);
                    char* base = reinterpret_cast<char*>(y + n);
                    const int4* ps = reinterpret_cast<const int4*>(my_slot + kCols * k);
                    const float4* pc = reinterpret_cast<const float4*>(my_scale + kCols * k);
                    auto all = [&](auto guard) {
#pragma unroll
                        for (int j = 0; j < kCols / 4; ++j) {
                            const int4 s4 = ps[j];
                            const float4 x4 = pc[j];
                            const int sl[4] = {s4.x, s4.y, s4.z, s4.w};
                            const float xc[4] = {x4.x, x4.y, x4.z, x4.w};
                            float r[4];
#pragma unroll
                            for (int i = 0; i < 4; ++i) r[i] = v[4 * j + i] * wn.near * xc[i];
                            if (rest) {
#pragma unroll
                                for (int i = 0; i < 4; ++i) r[i] *= wn.rest;
                            }
#pragma unroll
                            for (int i = 0; i < 4; ++i)
                                if (!decltype(guard)::value || (unsigned)sl[i] < (unsigned)slots)
                                    *reinterpret_cast<Y*>(base + (uint64_t)(uint32_t)sl[i] * row) = to_type<Y>(r[i]);
                        }
                    };
                    if (!grouped && kCols * k + kCols <= un.n) all(std::false_type());
                    else all(std::true_type());
                }
            };
            auto put = [&](int k, const float v[kCols]) {
                if (PX == 2) put_as(c.op == P_DOWN || p.ks > 1 ? p.part + (long long)un.split * c.M * w.N : static_cast<float*>(c.y), k, v);
                else if (c.op == P_DOWN || p.ks > 1) put_as(p.part + (long long)un.split * c.M * w.N, k, v);
                else if (c.xt == X_F16) put_as(static_cast<__half*>(c.y), k, v);
                else put_as(static_cast<__nv_bfloat16*>(c.y), k, v);
            };
            auto release = [&](int ab) {
                __syncwarp();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) {
                    if (CG == 2) mbar_arrive_cluster(leader_addr(smem_u32(&acc_empty[ab])));
                    else mbar_arrive(smem_u32(&acc_empty[ab]));
                }
            };
            constexpr int kSums = PX == 2 ? kQgBX2 / kCols / kQgEpiHalves : 1;
            float sum[kSums][kCols];
            for (int c0 = un.j0; c0 < un.j1; c0 += chunk, ++cc) {
                const int ab = p.nacc == 2 ? (cc & 1) : 0, use = p.nacc == 2 ? (cc >> 1) : cc;
                if (!(ok = qg_wait_warp(smem_u32(&acc_full[ab]), (uint32_t)(use & 1), false, flags, p.err))) break;
                tc_fence_after();
                __syncwarp();
                const uint32_t acol = tmem + tq + (uint32_t)(ab * p.accw);
                if (PX == 2) {
#pragma unroll
                    for (int k = 0; k < kSums; k += 2) {
                        uint32_t r[2][kCols] = {};
#pragma unroll
                        for (int h = 0; h < 2; ++h)
                            if (half + kQgEpiHalves * (k + h) < nch) tc_ld8(acol + kCols * (half + kQgEpiHalves * (k + h)), r[h]);
                        tc_wait_ld();
                        if (k + 2 >= kSums) release(ab);
#pragma unroll
                        for (int h = 0; h < 2; ++h)
#pragma unroll
                            for (int i = 0; i < kCols; ++i) {
                                asm volatile("" : "+r"(r[h][i]));  // not used before the wait
                                float& to = sum[PX == 2 ? k + h : 0][i];
                                to = c0 == un.j0 ? __uint_as_float(r[h][i]) : to + __uint_as_float(r[h][i]);
                            }
                    }
                } else {
                    uint32_t r[kCols];
                    if (half < nch) tc_ld8(acol + kCols * half, r);
                    for (int k = half; k < nch; k += kQgEpiHalves) {
                        tc_wait_ld();
                        float v[kCols];
#pragma unroll
                        for (int i = 0; i < kCols; ++i) v[i] = __uint_as_float(r[i]);
                        if (k + kQgEpiHalves < nch) tc_ld8(acol + kCols * (k + kQgEpiHalves), r);
                        put(k, v);
                    }
                    release(ab);
                }
            }
            if (!ok) break;
            if (PX == 2) {
                // one copy of the code: four side by side do not fit the registers
#pragma unroll 1
                for (int k = half; k < nch; k += kQgEpiHalves) {
                    put(k, sum[0]);
#pragma unroll
                    for (int j = 0; j + 1 < kSums; ++j)
#pragma unroll
                        for (int i = 0; i < kCols; ++i) sum[j][i] = sum[j + 1][i];
                }
            }
        }
        cp_async_wait<0>();  // after a wait that gave up, the next tables are still on their way
    } else {
        // ------------------------------ conversion ------------------------------
        const int cw = warp - kQgConv0, q = warp & 3, hh = (cw >> 2) & 1, grp = cw >> 3;  // row block 2 q + hh of a tile
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
        const uint32_t magic = opaque(0x64006400u);
        bool ok = true;
        // 2^-a of rows g, g + 8, asked for a unit ahead
        float is0 = 1.0f, is1 = 1.0f;
        auto ask = [&](const QgUnit& un) {
            const float* is = p.wis + ((long long)un.e * w.RB + min(8 * un.nt + 2 * q + hh, w.RB - 1)) * 16 + (lane >> 2);
            is0 = __ldg(is);
            is1 = __ldg(is + 8);
        };
        QgUnit un = {}, un_next = {};
        if (first_unit < units) {
            un_next = place(first_unit, 0);
            ask(un_next);
        }
        for (int u = first_unit, ui = 0; u < units && ok; u += unit_step, ++ui) {
            un = un_next;
            const float m0 = __frcp_rn(is0), m1 = __frcp_rn(is1);
            if (u + unit_step < units) {
                un_next = place(u + unit_step, ui + 1);
                ask(un_next);
            }
            // The groups take tiles in turn, whatever a unit's number of them: a group that waits for
            // the release of tile t - nstage has waited for t - groups - nstage, so that with nstage >=
            // groups the stage's barrier is at most one phase behind the wait's parity.
            for (int j = un.j0; j < un.j1; ++j, turn = turn + 1 == kQgGroups ? 0 : turn + 1) {
                const QgRing at = g, ar = r;
                g.next(p.nstage);
                r.next(p.nraw);
                if (turn != grp) continue;
                if (!(ok = qg_wait_warp(smem_u32(&r_full[ar.s]), ar.ph, r_ready, flags, p.err))) break;
                // tested here, needed after the conversion
                const uint32_t e_ready = mbar_test(smem_u32(&empty[at.s]), at.ph ^ 1u);
                const uint8_t* seg = raw(ar.s) + (2 * q + hh) * seg_bytes;
                const uint32_t col = tmem + ((uint32_t)(32 * q + 16 * hh) << 16) + (uint32_t)(p.nacc * p.accw + 64 * PA * at.s);
                // what needs no free stage comes before the wait for one, and before the last
                // tile's stores are waited for
                // with two pieces half of a 64-K tile's registers at a time: all of them were spilled
                constexpr int kWords = PA == 1 ? 4 : 2, kSteps = 8 / kWords;
                uint32_t hi[4 * kWords], lo[4 * kWords];
                QgGroup gc;
                uint4 codes = reinterpret_cast<const uint4*>(seg)[lane];
                qg_convert<PA, NG, kWords>(seg, codes, 0, 0, lane, magic, m0, m1, gc, hi, lo);
                announce();
                if (!(ok = qg_wait_warp(smem_u32(&empty[at.s]), at.ph ^ 1u, e_ready, flags, p.err))) break;
                QgRing rn = r;  // this group's next raw stage
                rn.skip(kQgGroups - 1, p.nraw);
                r_ready = mbar_test(smem_u32(&r_full[rn.s]), rn.ph);
                tc_fence_after();
                __syncwarp();
#pragma unroll
                for (int step = 0; step < kSteps; ++step) {
                    if (step > 0) {
                        if (step * 2 == kSteps) codes = reinterpret_cast<const uint4*>(seg + kQgTile)[lane];
                        qg_convert<PA, NG, kWords>(seg, codes, step * 2 / kSteps, step * kWords % 4, lane, magic, m0, m1, gc, hi, lo);
                        if (step == kSteps - 1) {
                            __syncwarp();
                            if (lane == 0) mbar_arrive(smem_u32(&r_empty[ar.s]));
                        }
                    }
                    tc_st_frag<4 * kWords>(col + 8 * kWords * step, hi);
                    if (PA == 2) tc_st_frag<4 * kWords>(col + 64 + 8 * kWords * step, lo);
                }
                stored = at.s;
                if (p.nstage <= kQgGroups) announce();  // no stage to spare
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

}  // namespace qmm
