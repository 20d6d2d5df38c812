// qmm_moe_layer.cuh -- a whole mixture-of-experts layer for a few tokens in two
// launches.
//
// Mathematics: that of the four calls that it stands for.  l = x R^T in f32;
// the routing of qmm_moe_route.cu; h = silu(x Wg^T) (x Wu^T) of each token's
// experts, rounded to the activations' type; y = sum_j p_j (h_j Wd^T).
//
// A decode step's layer reads a few MB of weights per SM's share, so what
// stands between the products is what costs: a launch, its ramp and its tail
// each time.  The first launch forms the logits (a block per expert).  In the
// second every block routes all tokens for itself (some microseconds of one
// warp a token, no exchange), then takes shares of the work by tickets: first
// the shares of the experts' first products, then those of the second ones,
// which wait until all of the first are reported, and with more than a token an
// item those of the tokens' sums.  A ticket's holder runs already when it waits,
// and what it waits for are shares with lower tickets, whose holders do not wait
// for it: however few blocks are on the GPU at a time, the layer ends.  The
// weights of a second product are on their way before its block waits, as the
// experts are known.  The products themselves are the row kernel's
// (qmm_q4g_rows.cuh, qg_rows_share).
//
// Waits are bounded: one that gives up raises the error word and its block ends.
#pragma once

#include "qmm_moe_route.cuh"
#include "qmm_q4g_rows.cuh"

namespace qmm {

constexpr int kMoeWarps = 16, kMoeThreads = kMoeWarps * 32;

struct MoeParams {
    RouteParams route;   // c.ids, c.weights: for the caller, or NULL
    QgRowsParams up, down;
    unsigned* counters;  // [0] tickets, [1] shares of the first products done, [2] of the second
    unsigned* err;
    int epl16;           // experts per lane in the routing: 16, or 4
    int off_route;
    int stall;
};

__device__ __forceinline__ unsigned ld_acquire(const unsigned* p) {
    unsigned v;
    asm volatile("ld.acquire.gpu.global.u32 %0, [%1];" : "=r"(v) : "l"(p) : "memory");
    return v;
}
__device__ __forceinline__ void add_release(unsigned* p) { asm volatile("red.release.gpu.global.add.u32 [%0], 1;" ::"l"(p) : "memory"); }

// Waits until *p is n; called by one thread.
static __device__ __noinline__ bool moe_wait(const unsigned* p, unsigned n, unsigned* err) {
    const long long t0 = clock64();
    long long lim = 0;
    while (ld_acquire(p) != n) {
        const long long dt = clock64() - t0;
        if (dt <= kWaitLimitCheck) continue;
        if (lim == 0) lim = wait_limit(err);
        if (dt > lim) {
            atomicOr(err, ERR_TIMEOUT);
            return false;
        }
        __nanosleep(100);
    }
    return true;
}

// The rows of a product that others' shares make: waited for once.
struct MoeWait {
    const unsigned* done;  // NULL: nothing to wait for
    unsigned n;
    unsigned* err;
    int* s_ok;
    __device__ __forceinline__ void route() {}
    __device__ __forceinline__ bool rows() {
        if (!done) return true;
        if (threadIdx.x == 0) *s_ok = moe_wait(done, n, err);
        __syncthreads();
        done = nullptr;
        return *s_ok != 0;
    }
};

template <int NB, bool BF, bool TOKEN>
__global__ void __launch_bounds__(kMoeThreads, 1) moe_layer_kernel(const __grid_constant__ MoeParams p) {
    extern __shared__ __align__(16) uint8_t sm[];
    __shared__ int s_e[kQgMaxK];
    __shared__ float s_wt[kQgMaxK];
    __shared__ int s_row[64];
    __shared__ int ts_up[kQgRowMaxE + 1], ts_down[kQgRowMaxE + 1];
    __shared__ int s_ok;
    __shared__ unsigned s_ticket[2];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int T = p.route.c.T, E = p.route.c.E, k = p.route.c.top_k, S = T * k;
    int* ids = reinterpret_cast<int*>(sm + p.off_route);      // [S]
    float* weights = reinterpret_cast<float*>(ids + S);       // [S]
    int* order = reinterpret_cast<int*>(weights + S);         // [S]
    int* offsets = order + S;                                 // [E + 1]
    uint32_t* mask = reinterpret_cast<uint32_t*>(offsets + E + 1);  // [E] the tokens that chose an expert
    for (int e = tid; e < E; e += kMoeThreads) mask[e] = 0u;
    grid_dep_launch();
    __syncthreads();
    grid_dep_wait();
    unsigned next = 0;  // thread 0: the next ticket
    if (tid == 0) next = atomicAdd(p.counters, 1u);

    // ------------------------------ routing ------------------------------
    RouteParams rp = p.route;
    rp.c.ids = ids;
    rp.c.weights = weights;
    uint32_t* picks = reinterpret_cast<uint32_t*>(sm) + warp * E;  // where the products' rings will be
    for (int t = warp; t < T; t += kMoeWarps) {
        const int id = p.epl16 ? route_token<16>(rp, t, picks, lane) : route_token<4>(rp, t, picks, lane);
        if (lane < k) atomicOr(&mask[id], 1u << t);
    }
    __syncthreads();
    const bool by_expert = !TOKEN || !p.up.by_slot;
    if (by_expert && warp == 0) {
        // slots sorted by expert, by token within one: a count is a mask's population, a rank that of its lower bits
        const int per = (E + 31) / 32;
        int mine = 0;
        for (int i = 0; i < per; ++i)
            if (lane * per + i < E) mine += __popc(mask[lane * per + i]);
        int pre = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int u = __shfl_up_sync(0xffffffffu, pre, o);
            if (lane >= o) pre += u;
        }
        if (lane == 31) offsets[E] = pre;
        pre -= mine;
        for (int i = 0; i < per; ++i) {
            const int e = lane * per + i;
            if (e >= E) break;
            offsets[e] = pre;
            pre += __popc(mask[e]);
        }
        __syncwarp();
        for (int s = lane; s < S; s += 32) {
            const int t = s / k, e = ids[s];
            order[offsets[e] + __popc(mask[e] & ((1u << t) - 1u))] = s;
        }
        __syncwarp();
        if (!p.up.by_slot) qg_rows_items(offsets, E, S, p.up.cols, ts_up, lane);
        if (!TOKEN) qg_rows_items(offsets, E, S, p.down.cols, ts_down, lane);
    }
    if (blockIdx.x == 0 && p.route.c.ids)
        for (int s = tid; s < S; s += kMoeThreads) {
            p.route.c.ids[s] = ids[s];
            p.route.c.weights[s] = weights[s];
        }

    // ------------------------------ shares ------------------------------
    const unsigned G = gridDim.x, total = TOKEN ? 2 * G : 3 * G;
    for (int it = 0;; ++it) {
        if (tid == 0) s_ticket[it & 1] = next;
        __syncthreads();  // and what the last share kept in shared memory is no longer read
        const unsigned ticket = s_ticket[it & 1];
        if (ticket >= total) break;
        if (tid == 0) next = atomicAdd(p.counters, 1u);
        const unsigned phase = ticket / G, i = ticket - phase * G;
        if (phase == 2) {
            // a token's second products, in the order of its choices
            if (tid == 0) s_ok = moe_wait(p.counters + 2, G, p.err);
            __syncthreads();
            if (!s_ok) break;
            const QgCall& c = p.down.c;
            const int N = c.w.N;
            const long long n = (long long)T * N, o1 = (long long)(i + 1) * n / G;
            for (long long o = (long long)i * n / G + tid; o < o1; o += kMoeThreads) {
                const int t = (int)(o / N), col = (int)(o - (long long)t * N);
                float v = 0.0f;
#pragma unroll 8
                for (int j = 0; j < k; ++j) v = fmaf(weights[t * k + j], __ldcg(p.down.part + (long long)(t * k + j) * N + col), v);
                x_store(c.y, c.xt, o, v);
            }
            continue;
        }
        const bool second = phase == 1;
        const QgRowsParams& q = second ? p.down : p.up;
        const int* ts = second ? ts_down : ts_up;
        const long long items = second ? (TOKEN ? T : ts[E]) : q.by_slot ? S : ts[E];
        const long long work = items * q.c.w.RB, w0 = i * work / G, w1 = (i + 1) * work / G;
        const QgRowsShared sh = {s_e, s_wt, s_row, ts, ids, weights, offsets, order};
        MoeWait wait = {second ? p.counters + 1 : nullptr, G, p.err, &s_ok};
        if (tid == 0) {
            s_ok = 1;
            *reinterpret_cast<uint4*>(sm + q.off_zero) = make_uint4(0u, 0u, 0u, 0u);  // what lanes without a column read
        }
        if (second) {
            if (q.c.w.ng == 1) qg_rows_share<TOKEN ? 1 : NB, BF, 1, TOKEN>(q, sm, sh, w0, w1, wait);
            else if (q.c.w.ng == 2) qg_rows_share<TOKEN ? 1 : NB, BF, 2, TOKEN>(q, sm, sh, w0, w1, wait);
            else qg_rows_share<TOKEN ? 1 : NB, BF, 4, TOKEN>(q, sm, sh, w0, w1, wait);
        } else {
            if (q.c.w.ng == 1) qg_rows_share<NB, BF, 1, false>(q, sm, sh, w0, w1, wait);
            else if (q.c.w.ng == 2) qg_rows_share<NB, BF, 2, false>(q, sm, sh, w0, w1, wait);
            else qg_rows_share<NB, BF, 4, false>(q, sm, sh, w0, w1, wait);
        }
        cp_async_wait<0>();
        __syncthreads();  // every thread's results are written
        if (!s_ok) break;
        if (tid == 0 && !(TOKEN && second) && !(p.stall && ticket == 0)) {
            __threadfence();
            add_release(p.counters + 1 + phase);
        }
    }
}

template <int NB, bool BF, bool TOKEN>
cudaError_t moe_layer_go(const MoePlan& pl, const MoeParams& p, int smem_max, cudaStream_t s) {
    static unsigned long long done = 0;
    auto* k = moe_layer_kernel<NB, BF, TOKEN>;
    const cudaError_t e = ensure_smem(k, smem_max - 8192, done);
    if (e != cudaSuccess) return e;
    return launch_pdl(k, (unsigned)pl.blocks, kMoeThreads, pl.smem, s, p);
}

}  // namespace qmm
