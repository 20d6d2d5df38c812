// qmm_q4g_rows.cu -- host side of the row kernel (its plan), and the kernel
// that adds the experts' partial rows of a token.
#include <cmath>

#include "qmm_q4g_rows.cuh"

namespace qmm {

cudaError_t launch_q4g_rows_1(const QgRowsPlan& pl, const QgRowsParams& p, int smem_max, cudaStream_t s);
cudaError_t launch_q4g_rows_2(const QgRowsPlan& pl, const QgRowsParams& p, int smem_max, cudaStream_t s);
cudaError_t launch_q4g_rows_4(const QgRowsPlan& pl, const QgRowsParams& p, int smem_max, cudaStream_t s);

namespace {

// Bound by the partial rows' bytes (4 top_k a value): eight independent loads a
// thread, V values wide.  Skipped slots have weight 0 and are not read.
template <int V>
__global__ void __launch_bounds__(256) q4g_combine_kernel(const float* __restrict__ part, QgRoute r, int E, int N, void* y, int xt) {
    grid_dep_launch();
    grid_dep_wait();
    const int t = blockIdx.x;
    const int n = (blockIdx.y * 256 + threadIdx.x) * V;
    if (n >= N) return;
    float v[V];
#pragma unroll
    for (int i = 0; i < V; ++i) v[i] = 0.0f;
    for (int j0 = 0; j0 < r.top_k; j0 += 8) {
        float wt[8], u[8][V];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const long long slot = (long long)t * r.top_k + j0 + j;
            bool on = j0 + j < r.top_k;
            if (on) {
                const int e = __ldg(r.ids + slot);
                on = e >= 0 && e < E;
            }
            wt[j] = on ? __ldg(r.weights + slot) : 0.0f;
            if (V == 4) {
                const float4 f = on ? __ldcg(reinterpret_cast<const float4*>(part + slot * N + n)) : make_float4(0.f, 0.f, 0.f, 0.f);
                u[j][0] = f.x;
                u[j][1 % V] = f.y;
                u[j][2 % V] = f.z;
                u[j][3 % V] = f.w;
            } else {
                u[j][0] = on ? __ldcg(part + slot * N + n) : 0.0f;
            }
        }
#pragma unroll
        for (int j = 0; j < 8; ++j)
#pragma unroll
            for (int i = 0; i < V; ++i) v[i] = fmaf(wt[j], u[j][i], v[i]);
    }
#pragma unroll
    for (int i = 0; i < V; ++i) x_store(y, xt, (long long)t * N + n + i, v[i]);
}

// four loads in flight a thread
__global__ void __launch_bounds__(256) q4g_sum_kernel(const float* __restrict__ part, int ks, long long n, void* y, int xt) {
    grid_dep_launch();
    grid_dep_wait();
    const long long i = (long long)blockIdx.x * 256 + threadIdx.x;
    if (i >= n) return;
    float v = 0.0f;
    for (int s0 = 0; s0 < ks; s0 += 4) {
        float u[4];
#pragma unroll
        for (int s = 0; s < 4; ++s) u[s] = s0 + s < ks ? __ldcg(part + (s0 + s) * n + i) : 0.0f;
#pragma unroll
        for (int s = 0; s < 4; ++s) v += u[s];
    }
    x_store(y, xt, i, v);
}

}  // namespace

cudaError_t launch_q4g_sum(const float* part, int ks, long long n, void* y, int xt, cudaStream_t s) {
    return launch_pdl(q4g_sum_kernel, (unsigned)((n + 255) / 256), 256, 0, s, part, ks, n, y, xt);
}

cudaError_t launch_q4g_combine(const float* part, const QgRoute& r, int E, int N, void* y, int xt, cudaStream_t s) {
    const int V = N % 4 == 0 ? 4 : 1;  // rows that start on 16 bytes
    const unsigned gy = (unsigned)((N / V + 255) / 256);
    return V == 4 ? launch_pdl_2d(q4g_combine_kernel<4>, (unsigned)r.T, gy, 256, 0, s, part, r, E, N, y, xt)
                  : launch_pdl_2d(q4g_combine_kernel<1>, (unsigned)r.T, gy, 256, 0, s, part, r, E, N, y, xt);
}

QgRowsPlan plan_q4g_rows(const QgCall& c, int sms, int smem_max) {
    QgRowsPlan pl;
    pl.np = c.xt == X_F32 ? 3 : 1;
    if (c.op != P_DENSE && c.w.E > kQgRowMaxE) return pl;
    const long long row_bytes = (long long)pl.np * c.w.KS * kQgSegK * 2;  // staged bytes of one activation row
    const long long slots = c.M;
    if (c.op != P_DENSE) {
        // one slot (one token) an item while few slots share an expert: no items to look up, and no
        // partial sums; by expert, an item is up to `cols` of its slots with one weight stream
        pl.by_slot = c.r.T <= 4 && c.r.top_k <= kQgMaxK && (c.op == P_GATE_UP || row_bytes * c.r.top_k <= 96 * 1024);
    }
    const bool token = c.op == P_DOWN && pl.by_slot;
    const long long rows_mul = token ? c.r.top_k : 1;
    const int seg = qg_seg_bytes(c.w.ng), VS = (int)(c.w.KS * rows_mul);
    auto nb_of = [&](int cols) { const int b = (cols * pl.np + 7) / 8; return b <= 1 ? 1 : b <= 2 ? 2 : 4; };
    auto red = [&](int nb, int warps) { return 2ll * warps * nb * 128 * 4; };
    // shared memory: activations, the warps' sums, their rings
    auto need = [&](int cols, int warps) {
        return cols * row_bytes * rows_mul + 16 + red(nb_of(cols), warps) + (long long)warps * kQgDepth * seg;
    };
    const long long room = smem_max - kQgRowStatic - 1024;
    // Rows of x per item: full MMA column blocks, or what there is.  A second block of columns costs
    // a segment about half as much again, four about 1.3 times as much again.
    int choices[3] = {8 / pl.np, 16 / pl.np, 32 / pl.np}, nchoice = 3;
    if (c.op != P_DENSE) {
        const long long avg = (slots + c.w.E - 1) / c.w.E;
        choices[0] = pl.by_slot ? 1 : avg * pl.np <= 4 ? 8 / pl.np : avg * pl.np <= 8 ? 16 / pl.np : 32 / pl.np;
        nchoice = 1;
    }
    double best = 0;
    for (int ch = 0; ch < nchoice; ++ch) {
        int cols = c.op == P_DENSE && c.M < choices[ch] ? c.M : choices[ch];
        while (cols > 1 && need(cols, 8) > room) --cols;  // as many as shared memory holds beside eight warps
        if (need(cols, 8) > room) continue;
        long long items;  // expected
        if (c.op == P_DENSE) {
            items = (c.M + cols - 1) / cols;
            cols = (int)((c.M + items - 1) / items);
        } else if (pl.by_slot) {
            items = c.op == P_GATE_UP ? slots : c.r.T;
        } else {
            // the experts that some slot chose, under even routing; an expert's last item may be partial
            items = (long long)(c.w.E * (1.0 - pow(1.0 - 1.0 / c.w.E, (double)slots)) + 0.999) + slots / cols;
            if (items > c.w.E + slots / cols) items = c.w.E + slots / cols;
            if (items > slots) items = slots;
        }
        if (items < 1) items = 1;
        const int nb = nb_of(cols);
        for (int warps : {24, 16, 8}) {
            if (warps > qg_row_warps(nb) || need(cols, warps) > room) continue;
            for (int wk = 1; wk <= 8; wk *= 2) {
                const int wr = warps / wk, nit = (VS + wk - 1) / wk;
                if (wr > 15 && wk > 1) continue;  // named barriers
                const long long work = items * c.w.RB, blocks = work < sms ? work : sms;
                const double share = (double)work / blocks;  // row blocks per block
                // segments a warp takes in turn, its row blocks' barriers and sums (about one each);
                // more warps share an SM's issue slots
                const double cost = ceil(share / wr) * (nit + 1.0) * (warps >= 16 ? warps / 16.0 : 1.0) * (nb == 1 ? 1.0 : nb == 2 ? 1.5 : 2.3);
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
    pl.smem = (size_t)need(pl.cols, pl.warps);
    pl.off_zero = (int)(pl.cols * row_bytes * rows_mul);
    pl.off_red = pl.off_zero + 16;
    pl.off_ring = pl.off_red + (int)red(pl.nb, pl.warps);
    if (c.op == P_DOWN && !pl.by_slot) pl.workspace = (size_t)slots * c.w.N * 4;
    pl.ok = true;
    return pl;
}

cudaError_t launch_q4g_rows(const QgRowsPlan& pl, const QgCall& c, void* ws, int smem_max, cudaStream_t s) {
    QgRowsParams p;
    p.c = c;
    p.part = static_cast<float*>(ws);
    p.by_slot = pl.by_slot;
    p.cols = pl.cols;
    p.np = pl.np;
    p.wk = pl.wk;
    p.wr = pl.warps / pl.wk;
    p.wk_log2 = pl.wk == 1 ? 0 : pl.wk == 2 ? 1 : pl.wk == 4 ? 2 : 3;
    p.off_zero = pl.off_zero;
    p.off_red = pl.off_red;
    p.off_ring = pl.off_ring;
    cudaError_t e = pl.nb == 1   ? launch_q4g_rows_1(pl, p, smem_max, s)
                    : pl.nb == 2 ? launch_q4g_rows_2(pl, p, smem_max, s)
                                 : launch_q4g_rows_4(pl, p, smem_max, s);
    if (e != cudaSuccess || c.op != P_DOWN || pl.by_slot) return e;
    return launch_q4g_combine(p.part, c.r, c.w.E, c.w.N, c.y, c.xt, s);
}

}  // namespace qmm
