// qmm_q4g_gemm.cu -- host side of the 4-bit group-scale GEMM: plan,
// activation preparation, launches.
#include "qmm_q4g_gemm.cuh"

namespace qmm {
namespace {

// One row per block: f16 values (pieces) scaled by 2^b, and 2^-b.  The scale
// comes from the row's largest finite magnitude; infinities and NaN stay what
// they are (their rests are 0).  For experts row p is the activations of slot
// order[p].
template <int NP>
__global__ void __launch_bounds__(256) q4g_prep_kernel(const QgCall c, int rows, __half* out, float* xs) {
    __shared__ float red[8];
    grid_dep_launch();
    grid_dep_wait();
    const int row = blockIdx.x, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, K = c.w.K, xt = c.xt;
    const void* x = c.x;
    int from = row;
    if (c.op != P_DENSE) {
        if (row >= c.r.offsets[c.w.E]) return;
        from = c.r.order[row];
        if (from < 0 || from >= rows) return;
        if (c.op == P_GATE_UP) from /= c.r.top_k;
    }
    const long long at = (long long)from * c.ldx;
    if (xt == X_F16) {
        for (int k = 8 * tid; k < K; k += 8 * 256)
            *reinterpret_cast<uint4*>(out + (long long)row * K + k) = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(x) + at + k);
        return;
    }
    auto load8 = [&](int k, float f[8]) {
        if (xt == X_F32) {
            const float4 a = *reinterpret_cast<const float4*>(static_cast<const float*>(x) + at + k);
            const float4 b = *reinterpret_cast<const float4*>(static_cast<const float*>(x) + at + k + 4);
            f[0] = a.x; f[1] = a.y; f[2] = a.z; f[3] = a.w;
            f[4] = b.x; f[5] = b.y; f[6] = b.z; f[7] = b.w;
        } else {
            const uint4 u = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(x) + at + k);
            const uint32_t v[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                f[2 * j] = __uint_as_float(v[j] << 16);
                f[2 * j + 1] = __uint_as_float(v[j] & 0xffff0000u);
            }
        }
    };
    float m = 0.0f;
    for (int k = 8 * tid; k < K; k += 8 * 256) {
        float f[8];
        load8(k, f);
#pragma unroll
        for (int j = 0; j < 8; ++j) m = fabsf(f[j]) < INFINITY ? fmaxf(m, fabsf(f[j])) : m;
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    if (lane == 0) red[warp] = m;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 8; ++i) m = fmaxf(m, red[i]);
    const float is = tc_row_iscale(m), sc = __frcp_rn(is);
    if (tid == 0) xs[row] = is;
    for (int k = 8 * tid; k < K; k += 8 * 256) {
        float f[8];
        load8(k, f);
        uint32_t h[4], l[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const float a = f[2 * j] * sc, b = f[2 * j + 1] * sc;
            const __half2 v = __floats2half2_rn(a, b);
            h[j] = *reinterpret_cast<const uint32_t*>(&v);
            if (NP == 2) {
                const float2 vf = __half22float2(v);
                const __half2 r = __floats2half2_rn(fabsf(a) < INFINITY ? a - vf.x : 0.0f, fabsf(b) < INFINITY ? b - vf.y : 0.0f);
                l[j] = *reinterpret_cast<const uint32_t*>(&r);
            }
        }
        *reinterpret_cast<uint4*>(out + (long long)row * K + k) = make_uint4(h[0], h[1], h[2], h[3]);
        if (NP == 2) *reinterpret_cast<uint4*>(out + ((long long)rows + row) * K + k) = make_uint4(l[0], l[1], l[2], l[3]);
    }
}

template <int NP, int NG>
cudaError_t gemm_one(const QgGemmPlan& pl, const CUtensorMap& tx, const QgGemmParams& p, int smem_max, cudaStream_t s) {
    static unsigned long long done = 0;
    auto* k = q4g_gemm_kernel<NP, NG>;
    const cudaError_t e = ensure_smem(k, smem_max, done);
    if (e != cudaSuccess) return e;
    return launch_pdl(k, (unsigned)pl.grid, kQgThreads, pl.smem, s, tx, p);
}

}  // namespace

QgGemmPlan plan_q4g_gemm(const QgCall& c, int sms, int smem_max) {
    QgGemmPlan pl;
    const bool grouped = c.op != P_DENSE;
    if (grouped && c.w.E > kQgMaxE) return pl;
    const long long rows = c.M;
    pl.np = c.xt == X_F32 ? 2 : 1;
    pl.prep = grouped || c.xt != X_F16;
    const long long per = grouped ? (c.M + c.w.E - 1) / c.w.E : c.M;  // activation rows per weight matrix
    pl.ntiles = (c.w.RB + 7) / 8;
    // tiles of 256 rows amortise the weights' conversion best; two accumulators of 128 columns
    // let the epilogue run beside the next unit's MMAs
    const int most = pl.np == 2 ? 128 : 256;
    if (grouped) {
        pl.bx = per >= 192 && most == 256 ? 256 : per > 48 ? 128 : per > 24 ? 64 : 32;
    } else {
        const int tiles = (int)((per + most - 1) / most);
        pl.bx = (int)((per + tiles - 1) / tiles + 15) / 16 * 16;
    }
    pl.box = grouped && pl.bx > 64 ? 64 : pl.bx;  // an expert's tile is any size: no more copied than 63 rows too many
    pl.nacc = pl.bx <= 128 ? 2 : 1;
    pl.mtiles = grouped ? 0 : (int)((per + pl.bx - 1) / pl.bx);
    pl.nraw = 3;
    const int raw = 16 * qg_seg_bytes(c.w.ng), stage = pl.bx * 128 * pl.np;
    const int fixed = 512 + 2 * 8 * 128 * 4 + (c.w.E + 1) * 4 + 1024;
    pl.nstage = (smem_max - fixed - pl.nraw * raw) / stage;
    const int cap = 8 / pl.np;
    if (pl.nstage > cap) pl.nstage = cap;
    if (pl.nstage < 2) return pl;
    pl.smem = (size_t)pl.nstage * stage + (size_t)pl.nraw * raw + fixed;
    const long long units = grouped ? ((long long)c.w.E + c.M / pl.bx) * pl.ntiles : (long long)pl.mtiles * pl.ntiles;
    if (units > (1ll << 30)) return pl;
    pl.grid = (int)(units < sms ? units : sms);
    auto r256 = [](size_t v) { return (v + 255) / 256 * 256; };
    pl.ws_x = 0;
    pl.ws_xs = pl.prep ? r256((size_t)pl.np * rows * c.w.K * 2) : 0;
    pl.ws_part = pl.ws_xs + (pl.prep ? r256((size_t)rows * 4) : 0);
    pl.workspace = pl.ws_part + (c.op == P_DOWN ? (size_t)c.M * c.w.N * 4 : 0);
    pl.ok = true;
    return pl;
}

cudaError_t launch_q4g_gemm(const QgGemmPlan& pl, const QgCall& c, void* ws, unsigned* err, int smem_max, cudaStream_t s) {
    uint8_t* wsb = static_cast<uint8_t*>(ws);
    const int rows = c.M, K = c.w.K;
    const void* xsrc = c.x;
    long long pitch = c.ldx * 2;
    float* xs = nullptr;
    if (pl.prep) {
        __half* xh = reinterpret_cast<__half*>(wsb + pl.ws_x);
        if (c.xt != X_F16) xs = reinterpret_cast<float*>(wsb + pl.ws_xs);
        const cudaError_t e = pl.np == 2 ? launch_pdl(q4g_prep_kernel<2>, (unsigned)rows, 256, 0, s, c, rows, xh, xs)
                                         : launch_pdl(q4g_prep_kernel<1>, (unsigned)rows, 256, 0, s, c, rows, xh, xs);
        if (e != cudaSuccess) return e;
        xsrc = xh;
        pitch = (long long)K * 2;
    }
    CUtensorMap tx;
    if (!make_map(&tx, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, xsrc, (unsigned long long)K, (unsigned long long)rows * pl.np, (unsigned long long)pitch,
                  64, (unsigned)pl.box, CU_TENSOR_MAP_SWIZZLE_128B))
        return cudaErrorInvalidValue;
    QgGemmParams p;
    p.c = c;
    p.part = reinterpret_cast<float*>(wsb + pl.ws_part);
    p.xs = xs;
    p.wis = reinterpret_cast<const float*>(c.w.data + c.w.iscale_off);
    p.err = err;
    p.xrows = rows;
    p.bx = pl.bx;
    p.box = pl.box;
    p.nacc = pl.nacc;
    p.mtiles = pl.mtiles;
    p.ntiles = pl.ntiles;
    p.kt = (K + 63) / 64;
    p.nraw = pl.nraw;
    p.nstage = pl.nstage;
    p.grid = pl.grid;
    p.off_raw = pl.nstage * pl.bx * 128 * pl.np;
    p.off_bar = p.off_raw + pl.nraw * 16 * qg_seg_bytes(c.w.ng);
    cudaError_t e;
    if (pl.np == 2)
        e = c.w.ng == 1   ? gemm_one<2, 1>(pl, tx, p, smem_max, s)
            : c.w.ng == 2 ? gemm_one<2, 2>(pl, tx, p, smem_max, s)
                          : gemm_one<2, 4>(pl, tx, p, smem_max, s);
    else
        e = c.w.ng == 1   ? gemm_one<1, 1>(pl, tx, p, smem_max, s)
            : c.w.ng == 2 ? gemm_one<1, 2>(pl, tx, p, smem_max, s)
                          : gemm_one<1, 4>(pl, tx, p, smem_max, s);
    if (e != cudaSuccess || c.op != P_DOWN) return e;
    return launch_q4g_combine(p.part, c.r, c.w.E, c.w.N, c.y, c.xt, s);
}

}  // namespace qmm
