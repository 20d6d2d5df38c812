// qmm_q4g_gemm.cu -- host side of the 4-bit group-scale GEMM: plan,
// activation preparation, launches.
#include "qmm_q4g_gemm.cuh"

namespace qmm {
namespace {

// TPR threads per row (a warp where there are many, else a block): f16 values
// (pieces) scaled by 2^b, and 2^-b.  The scale comes from the row's largest
// finite magnitude; infinities and NaN stay what they are (their rests are 0).
// For experts row p is the activations of slot order[p], so that the GEMM's
// copies find an expert's rows in one piece.  Bound by the rows' bytes, mostly
// written and read again in L2 (16384 rows of 2048: 12 us); four 16-byte loads a
// lane are in flight.
template <int NP, int XT, int TPR>
__global__ void __launch_bounds__(256) q4g_prep_kernel(const QgCall c, int rows, __half* out, float* xs) {
    grid_dep_launch();
    grid_dep_wait();
    const int row = blockIdx.x * (256 / TPR) + threadIdx.x / TPR, lane = threadIdx.x % TPR, K = c.w.K, pitch = (K + 63) / 64 * 64;
    if (row >= rows) return;
    int from = row;
    if (c.op != P_DENSE) {
        if (row >= c.r.offsets[c.w.E]) return;
        from = c.r.order[row];
        if (from < 0 || from >= rows) return;
        if (c.op == P_GATE_UP) from /= c.r.top_k;
    }
    constexpr int V = XT == X_F32 ? 4 : 8;  // values in 16 bytes
    const uint4* x = reinterpret_cast<const uint4*>(static_cast<const uint8_t*>(c.x) + (long long)from * c.ldx * (16 / V));
    const int n = K / V;
    __half* hr = out + (long long)row * pitch;
    if (pitch != K && lane < 4) {  // the other half of the last 64 K
        reinterpret_cast<uint4*>(hr + K)[lane] = make_uint4(0u, 0u, 0u, 0u);
        if (NP == 2) reinterpret_cast<uint4*>(hr + (long long)rows * pitch + K)[lane] = make_uint4(0u, 0u, 0u, 0u);
    }
    if (XT == X_F16) {
        for (int i = lane; i < n; i += 4 * TPR) {
            uint4 v[4];
#pragma unroll
            for (int j = 0; j < 4; ++j)
                if (i + TPR * j < n) v[j] = __ldg(x + i + TPR * j);
#pragma unroll
            for (int j = 0; j < 4; ++j)
                if (i + TPR * j < n) reinterpret_cast<uint4*>(hr)[i + TPR * j] = v[j];
        }
        return;
    }
    auto unpack = [](const uint4& u, float f[8]) {
        const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            if (XT == X_F32) {
                f[j] = __uint_as_float(w[j]);
            } else {
                f[2 * j] = __uint_as_float(w[j] << 16);
                f[2 * j + 1] = __uint_as_float(w[j] & 0xffff0000u);
            }
        }
    };
    float m = 0.0f;
    for (int i = lane; i < n; i += 4 * TPR) {
        uint4 v[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) v[j] = i + TPR * j < n ? __ldg(x + i + TPR * j) : make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            float f[8];
            unpack(v[j], f);
#pragma unroll
            for (int e = 0; e < V; ++e) m = fabsf(f[e]) < INFINITY ? fmaxf(m, fabsf(f[e])) : m;
        }
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    if (TPR > 32) {
        __shared__ float red[8];
        if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = m;
        __syncthreads();
#pragma unroll
        for (int i = 0; i < 8; ++i) m = fmaxf(m, red[i]);
    }
    const float is = tc_row_iscale(m), sc = __frcp_rn(is);
    if (lane == 0) xs[row] = is;
    for (int i = lane; i < n; i += 4 * TPR) {
        uint4 v[4];
#pragma unroll
        for (int j = 0; j < 4; ++j)
            if (i + TPR * j < n) v[j] = __ldg(x + i + TPR * j);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            if (i + TPR * j >= n) continue;
            float f[8];
            unpack(v[j], f);
            uint32_t h[V / 2], l[V / 2];
#pragma unroll
            for (int e = 0; e < V / 2; ++e) {
                const float a = f[2 * e] * sc, b = f[2 * e + 1] * sc;
                const __half2 hv = __floats2half2_rn(a, b);
                h[e] = *reinterpret_cast<const uint32_t*>(&hv);
                if (NP == 2) {
                    const float2 vf = __half22float2(hv);
                    const __half2 r = __floats2half2_rn(fabsf(a) < INFINITY ? a - vf.x : 0.0f, fabsf(b) < INFINITY ? b - vf.y : 0.0f);
                    l[e] = *reinterpret_cast<const uint32_t*>(&r);
                }
            }
            if constexpr (V == 8) {
                reinterpret_cast<uint4*>(hr)[i + TPR * j] = make_uint4(h[0], h[1], h[2], h[3]);
            } else {
                reinterpret_cast<uint2*>(hr)[i + TPR * j] = make_uint2(h[0], h[1]);
                reinterpret_cast<uint2*>(hr + (long long)rows * pitch)[i + TPR * j] = make_uint2(l[0], l[1]);
            }
        }
    }
}

template <int PA, int PX, int NG, int CG>
cudaError_t gemm_one(const QgGemmPlan& pl, const CUtensorMap& tx, const CUtensorMap& tw, const QgGemmParams& p, int smem_max, cudaStream_t s) {
    static unsigned long long done = 0;
    auto* k = q4g_gemm_kernel<PA, PX, NG, CG>;
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
    return cudaLaunchKernelEx(&cfg, k, tx, tw, p);
}

}  // namespace

QgGemmPlan plan_q4g_gemm(const QgCall& c, int sms, int smem_max) {
    QgGemmPlan pl;
    const bool grouped = c.op != P_DENSE;
    if (grouped && c.w.E > kQgMaxE) return pl;
    const long long rows = c.M;
    pl.np = c.xt == X_F32 ? 2 : 1;
    // f16 gate and up products: their weights' roundings would meet in the product of the two, 1.6
    // times the error of rounding the f16 output
    pl.pa = pl.np == 2 || (c.op == P_GATE_UP && c.xt == X_F16) ? 2 : 1;
    pl.prep = grouped || c.xt != X_F16 || c.w.K % 64 != 0;  // K that does not fill its last 64 is padded there
    const long long per = grouped ? (c.M + c.w.E - 1) / c.w.E : c.M;  // activation rows per weight matrix
    pl.cg = pl.np == 1 ? 2 : 1;
    pl.ntiles = (c.w.RB + 8 * pl.cg - 1) / (8 * pl.cg);
    const int workers = sms / pl.cg, unit = 16 * pl.cg;  // pairs; the MMA's N is a multiple of this
    // Modelled cycles (fitted to GB300 timings): a tile of 128 K costs its MMAs (half a cycle a
    // column, at least 40 each) or its conversion (900; two pieces 1400); a unit costs its
    // prologue and, where there is no second accumulator, the epilogue that the next unit's
    // MMAs wait for; slices of K cost their partial sums' traffic and a launch.
    const int most = pl.np == 2 ? kQgBX2 : pl.pa == 2 ? kQgBXA : kQgBX1;  // two pieces: the epilogue's running sums are registers
    pl.ks = 1;
    if (grouped) {
        // two accumulators: K is short, and a second one hides the epilogue (2048 tokens x 8 of 64,
        // 2048 -> 2 x 1024: 147 us with tiles of up to 192 rows, 153 with 160, 169 with 256)
        pl.bx = per > 96 ? (most < 192 ? most : 192) : per > 48 ? (most < 128 ? most : 128) : per > 24 ? 64 : 32;
    } else {
        double best = 0;
        for (int tiles = (int)((per + most - 1) / most); tiles <= 8 + (per + most - 1) / most; ++tiles) {
            const int bx = (int)((per + tiles - 1) / tiles + unit - 1) / unit * unit;
            const long long un = (long long)pl.ntiles * ((per + bx - 1) / bx);
            const double mma = 8.0 * (pl.pa + pl.np - 1) * (bx < 80 ? 40.0 : bx / 2.0), conv = pl.pa == 2 ? 1400.0 : 900.0, tile = mma > conv ? mma : conv;
            const double once = bx > 192 ? 1500.0 + 12.0 * bx : 1500.0;
            for (int ks = 1; ks <= c.w.KS && ks <= 16 && (ks == 1 || un * ks <= 2 * workers); ++ks) {
                const double waves = (double)((un * ks + workers - 1) / workers);
                const double cost = waves * ((double)((c.w.KS + ks - 1) / ks) * tile + once) + (ks > 1 ? 4000.0 + 8.0 * ks * per * c.w.N / 3000.0 : 0.0);
                if (best == 0 || cost < 0.98 * best) {
                    best = cost;
                    pl.bx = bx;
                    pl.ks = ks;
                }
            }
            if (bx == unit) break;
        }
    }
    pl.accw = (pl.bx + 31) / 32 * 32;
    pl.nacc = pl.bx <= 192 ? 2 : 1;  // with two accumulators the epilogue runs beside the next unit's MMAs
    pl.mtiles = grouped ? 0 : (int)((per + pl.bx - 1) / pl.bx);
    // converted weights in the tensor memory that the accumulators leave; activations and raw
    // weights share the shared memory
    pl.nstage = (kTcTmemCols - pl.nacc * pl.accw) / (64 * pl.pa);
    if (pl.nstage > kQgStageMax) pl.nstage = kQgStageMax;
    const int raw = 8 * qg_seg_bytes(c.w.ng), stage = pl.bx / pl.cg * 256 * pl.np;
    const int room = smem_max - (512 + 4 * kQgBX1 * 4 + (c.w.E + 1) * 8 + kQgTab * 16 + 1024);
    // Both rings are multiples of the converting groups, so that whoever waits for a stage's next
    // filling has waited for its last one (copies may land out of order).
    pl.nx = (room - 4 * raw) / stage / kQgGroups * kQgGroups;
    if (pl.nx > kQgXMax) pl.nx = kQgXMax;
    pl.nraw = (room - pl.nx * stage) / raw / kQgGroups * kQgGroups;
    if (pl.nraw > kQgRawMax) pl.nraw = kQgRawMax;
    if (pl.nstage < kQgGroups || pl.nx < kQgGroups || pl.nraw < kQgGroups) return pl;
    pl.smem = (size_t)pl.nx * stage + (size_t)pl.nraw * raw + (smem_max - room);
    const long long units = grouped ? ((long long)c.w.E + c.M / pl.bx) * pl.ntiles : (long long)pl.mtiles * pl.ntiles * pl.ks;
    if (units > (1ll << 30)) return pl;
    pl.grid = (int)(units < workers ? units : workers) * pl.cg;
    auto r256 = [](size_t v) { return (v + 255) / 256 * 256; };
    pl.ws_x = 0;
    pl.ws_xs = pl.prep ? r256((size_t)pl.np * rows * ((c.w.K + 63) / 64 * 64) * 2) : 0;
    pl.ws_part = pl.ws_xs + (pl.prep ? r256((size_t)rows * 4) : 0);
    pl.workspace = pl.ws_part + (c.op == P_DOWN || pl.ks > 1 ? (size_t)pl.ks * c.M * c.w.N * 4 : 0);
    pl.ok = true;
    return pl;
}

cudaError_t launch_q4g_gemm(const QgGemmPlan& pl, const QgCall& c, void* ws, unsigned* err, int stall, int smem_max, cudaStream_t s) {
    uint8_t* wsb = static_cast<uint8_t*>(ws);
    const int rows = c.M, K = c.w.K;
    const void* xsrc = c.x;
    long long pitch = c.ldx * 2;
    float* xs = nullptr;
    if (pl.prep) {
        __half* xh = reinterpret_cast<__half*>(wsb + pl.ws_x);
        if (c.xt != X_F16) xs = reinterpret_cast<float*>(wsb + pl.ws_xs);
        // a warp per row needs some 5000 rows to fill the GPU; a few rows take 9 us that way, 3 with a block each
        const bool many = rows >= 4096;
        const unsigned blocks = (unsigned)(many ? (rows + 7) / 8 : rows);
        auto* k = c.xt == X_F32   ? (many ? q4g_prep_kernel<2, X_F32, 32> : q4g_prep_kernel<2, X_F32, 256>)
                  : c.xt == X_F16 ? (many ? q4g_prep_kernel<1, X_F16, 32> : q4g_prep_kernel<1, X_F16, 256>)
                                  : (many ? q4g_prep_kernel<1, X_BF16, 32> : q4g_prep_kernel<1, X_BF16, 256>);
        const cudaError_t e = launch_pdl(k, blocks, 256, 0, s, c, rows, xh, xs);
        if (e != cudaSuccess) return e;
        xsrc = xh;
        pitch = (long long)(K + 63) / 64 * 64 * 2;
    }
    // activations: 64 K x rows x pieces x K / 64; a box has a block's rows (half a pair's), all
    // pieces and two of the last
    CUtensorMap tx;
    const unsigned long long xdims[4] = {64, (unsigned long long)rows, (unsigned long long)pl.np, (unsigned long long)(K + 63) / 64};
    const unsigned long long xstrides[3] = {(unsigned long long)pitch, (unsigned long long)pitch * rows, 128};
    const unsigned xbox[4] = {64, (unsigned)(pl.bx / pl.cg), (unsigned)pl.np, 2};
    if (!make_map_nd(&tx, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, xsrc, 4, xdims, xstrides, xbox, CU_TENSOR_MAP_SWIZZLE_128B)) return cudaErrorInvalidValue;
    // raw weights: row blocks of all experts, 8-byte elements, a box of a segment of eight of them
    CUtensorMap tw;
    const unsigned seg = (unsigned)qg_seg_bytes(c.w.ng);
    if (!make_map(&tw, CU_TENSOR_MAP_DATA_TYPE_UINT64, c.w.data, (unsigned long long)c.w.KS * (seg / 8), (unsigned long long)c.w.E * c.w.RB,
                  (unsigned long long)c.w.KS * seg, seg / 8, 8, CU_TENSOR_MAP_SWIZZLE_NONE))
        return cudaErrorInvalidValue;
    QgGemmParams p;
    p.c = c;
    p.part = reinterpret_cast<float*>(wsb + pl.ws_part);
    p.xs = xs;
    p.wis = reinterpret_cast<const float*>(c.w.data + c.w.iscale_off);
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
    p.stall = stall;
    p.stall_block = (unsigned)pl.cg - 1u;  // of a pair the second one, whose partner finds out by its own waits
    p.off_raw = pl.nx * (pl.bx / pl.cg) * 256 * pl.np;
    p.off_bar = p.off_raw + pl.nraw * 8 * qg_seg_bytes(c.w.ng);
    cudaError_t e;
    if (pl.np == 2)
        e = c.w.ng == 1   ? gemm_one<2, 2, 1, 1>(pl, tx, tw, p, smem_max, s)
            : c.w.ng == 2 ? gemm_one<2, 2, 2, 1>(pl, tx, tw, p, smem_max, s)
                          : gemm_one<2, 2, 4, 1>(pl, tx, tw, p, smem_max, s);
    else if (pl.pa == 2)
        e = c.w.ng == 1   ? gemm_one<2, 1, 1, 2>(pl, tx, tw, p, smem_max, s)
            : c.w.ng == 2 ? gemm_one<2, 1, 2, 2>(pl, tx, tw, p, smem_max, s)
                          : gemm_one<2, 1, 4, 2>(pl, tx, tw, p, smem_max, s);
    else
        e = c.w.ng == 1   ? gemm_one<1, 1, 1, 2>(pl, tx, tw, p, smem_max, s)
            : c.w.ng == 2 ? gemm_one<1, 1, 2, 2>(pl, tx, tw, p, smem_max, s)
                          : gemm_one<1, 1, 4, 2>(pl, tx, tw, p, smem_max, s);
    if (e == cudaSuccess && pl.ks > 1) return launch_q4g_sum(p.part, pl.ks, (long long)c.M * c.w.N, c.y, c.xt, s);
    if (e != cudaSuccess || c.op != P_DOWN) return e;
    return launch_q4g_combine(p.part, c.r, c.w.E, c.w.N, c.y, c.xt, s);
}

}  // namespace qmm
