// qmm_moe_route.cu -- routing of a mixture-of-experts layer: logits [T, E] to
// each token's top-k experts and weights, and the token slots sorted by expert.
//
// Mathematics.  score = softmax(l) or 1 / (1 + exp(-l)), in f32.  What is
// compared (the pick) is the logit itself for a softmax without bias (softmax
// keeps the order, and no rounding can change a choice), else the score plus
// the bias.  With groups, a group's value is its largest pick or the sum of
// its two largest; experts outside the best groups are out.  The k largest
// picks are taken in order; ties go to the lowest index.
//
// The work is a few operations per logit, so a small call is bound by latency
// and a large one by the selection's instructions.  One warp per token holds
// its picks in registers (expert lane + 32 i); a selection step is two
// warp-wide integer reductions (redux) on order-preserving keys, the second
// one settling ties.
//
// The order (a stable counting sort of the T k slots by expert) takes no
// atomics, so it is the same on every run: each block counts its tokens'
// slots by expert; in the second launch a block adds up the counts of all
// blocks (its own base positions and the offsets), and its warps rank their
// 32 consecutive slots at a time by matching lanes.  A call that fits one
// block does all of it in the first launch.
#include "qmm_q4g_internal.h"

namespace qmm {
namespace {

constexpr int kRouteWarps = 16;
constexpr int kRouteThreads = kRouteWarps * 32;


struct RouteParams {
    RouteCall c;
    int tile;      // tokens per block
    int blocks;
    unsigned* counts;  // [blocks][E] slots of each block by expert (more than one block)
};

// order-preserving integer key of a float; -0 counts as +0, NaN ranks below -inf; 0 is "none"
__device__ __forceinline__ uint32_t pick_key(float f) {
    if (f != f) return 1u;
    const uint32_t u = __float_as_uint(f + 0.0f);
    return u & 0x80000000u ? ~u : u | 0x80000000u;
}

// One token: EPL experts per lane.  sp: the warp's row of picks in shared memory (with groups).
template <int EPL>
__device__ __forceinline__ void route_token(const RouteCall& c, long long tok, float* sp, int lane) {
    float score[EPL];
    uint32_t key[EPL];
    const long long base = tok * c.ldl;
    float m = -INFINITY;
    // the type is told apart outside of the loads, so that they are in flight together
    if (c.xt == X_F32) {
#pragma unroll
        for (int i = 0; i < EPL; ++i) score[i] = lane + 32 * i < c.E ? static_cast<const float*>(c.logits)[base + lane + 32 * i] : -INFINITY;
    } else {
        uint16_t raw[EPL];
#pragma unroll
        for (int i = 0; i < EPL; ++i) raw[i] = lane + 32 * i < c.E ? static_cast<const uint16_t*>(c.logits)[base + lane + 32 * i] : (uint16_t)0;
#pragma unroll
        for (int i = 0; i < EPL; ++i)
            score[i] = lane + 32 * i >= c.E   ? -INFINITY
                       : c.xt == X_F16 ? __half2float(__ushort_as_half(raw[i]))
                                       : __uint_as_float((uint32_t)raw[i] << 16);
    }
#pragma unroll
    for (int i = 0; i < EPL; ++i) {
        if (score[i] != score[i]) score[i] = -INFINITY;  // a NaN logit is a masked one
        m = fmaxf(m, score[i]);
    }
    float total = 0.0f;
    if (!c.sigmoid) {
#pragma unroll
        for (int o = 16; o; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
#pragma unroll
        for (int i = 0; i < EPL; ++i) {
            const float l = score[i];
            // a row whose mask leaves nothing has no scores; l = m also covers +inf
            const float s = m == -INFINITY ? 0.0f : l == m ? 1.0f : expf(l - m);
            if (!c.bias) key[i] = pick_key(l);
            score[i] = lane + 32 * i < c.E ? s : 0.0f;
            total += score[i];
        }
#pragma unroll
        for (int o = 16; o; o >>= 1) total += __shfl_xor_sync(0xffffffffu, total, o);
        if (c.bias || !c.renorm) {
            const float d = total > 0.0f ? total : 1.0f;
#pragma unroll
            for (int i = 0; i < EPL; ++i) score[i] = score[i] / d;
        }
    } else {
#pragma unroll
        for (int i = 0; i < EPL; ++i) {
            score[i] = 1.0f / (1.0f + expf(-score[i]));
            if (!c.bias) key[i] = pick_key(score[i]);
        }
    }
    if (c.bias) {
#pragma unroll
        for (int i = 0; i < EPL; ++i) {
            const int e = lane + 32 * i;
            key[i] = pick_key(e < c.E ? score[i] + __ldg(c.bias + e) : 0.0f);
        }
    }
#pragma unroll
    for (int i = 0; i < EPL; ++i)
        if (lane + 32 * i >= c.E) key[i] = 0u;
    if (c.groups > 1) {
        // lanes per group: a power of two; lane r of group q takes its experts r, r + lpg, ...
        const int gs = c.E / c.groups;
        int lpg = 32;
        while (lpg * c.groups > 32) lpg >>= 1;
        uint32_t* sk = reinterpret_cast<uint32_t*>(sp);
        __syncwarp();
#pragma unroll
        for (int i = 0; i < EPL; ++i)
            if (lane + 32 * i < c.E) sk[lane + 32 * i] = key[i];
        __syncwarp();
        const int q = lane / lpg;
        uint32_t b1 = 0u, b2 = 0u;
        if (q < c.groups)
            for (int r = lane % lpg; r < gs; r += lpg) {
                const uint32_t k = sk[q * gs + r];
                b2 = max(b2, min(b1, k));
                b1 = max(b1, k);
            }
        for (int o = lpg >> 1; o; o >>= 1) {
            const uint32_t o1 = __shfl_xor_sync(0xffffffffu, b1, o), o2 = __shfl_xor_sync(0xffffffffu, b2, o);
            b2 = max(max(b2, o2), min(b1, o1));
            b1 = max(b1, o1);
        }
        uint32_t gk = b1;
        if (c.top2 && b2 != 0u) {
            const uint32_t u1 = b1 & 0x80000000u ? b1 & 0x7fffffffu : ~b1, u2 = b2 & 0x80000000u ? b2 & 0x7fffffffu : ~b2;
            gk = pick_key(__uint_as_float(u1) + __uint_as_float(u2));
        }
        if (q >= c.groups || lane % lpg != 0) gk = 0u;
        uint32_t kept = 0u;  // bit per group
        for (int s = 0; s < c.top_groups; ++s) {
            const uint32_t best = __reduce_max_sync(0xffffffffu, gk);
            const unsigned who = __ballot_sync(0xffffffffu, gk == best);
            const int l0 = __ffs(who) - 1;
            kept |= 1u << (l0 / lpg);
            if (lane == l0) gk = 0u;
        }
#pragma unroll
        for (int i = 0; i < EPL; ++i) {
            const int e = lane + 32 * i;
            if (e < c.E && !((kept >> (e / gs)) & 1u)) key[i] = 0u;
        }
    }
    // the k largest: lane j ends up with choice j
    int my_id = 0;
    float my_score = 0.0f, sum = 0.0f;
    for (int j = 0; j < c.top_k; ++j) {
        uint32_t b = 0u;
        int bi = 0;
#pragma unroll
        for (int i = 0; i < EPL; ++i)
            if (key[i] > b) {
                b = key[i];
                bi = i;
            }
        const uint32_t best = __reduce_max_sync(0xffffffffu, b);
        const uint32_t id = __reduce_min_sync(0xffffffffu, b == best ? (uint32_t)(lane + 32 * bi) : 0xffffffffu);
        float s = 0.0f;
#pragma unroll
        for (int i = 0; i < EPL; ++i) {
            const bool here = (int)id == lane + 32 * i;
            s = here ? score[i] : s;
            key[i] = here ? 0u : key[i];
        }
        s = __shfl_sync(0xffffffffu, s, (int)(id & 31u));
        sum += s;
        if (lane == j) {
            my_id = (int)id;
            my_score = s;
        }
    }
    if (lane < c.top_k) {
        const float v = c.renorm ? (sum > 0.0f ? my_score / sum : 0.0f) : my_score;
        c.ids[tok * c.top_k + lane] = my_id;
        c.weights[tok * c.top_k + lane] = c.scale == 1.0f ? v : v * c.scale;
    }
}

// exclusive prefix sum of a[0..n) in shared memory by the whole block, n <= 512; returns the total
__device__ __forceinline__ int block_scan(int* a, int n, int* tmp, int tid) {
    const int lane = tid & 31, warp = tid >> 5;
    int v = tid < n ? a[tid] : 0;
    int incl = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int u = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += u;
    }
    if (lane == 31) tmp[warp] = incl;
    __syncthreads();
    int before = 0, all = 0;
    for (int i = 0; i < kRouteWarps; ++i) {
        const int u = tmp[i];
        if (i < warp) before += u;
        all += u;
    }
    if (tid < n) a[tid] = before + incl - v;
    __syncthreads();
    return all;
}

// Counts the ids of slots [s0, s1) by expert, a row of `hist` [kRouteWarps][E]
// per warp; warp v has the v-th sixteenth of the 32-slot steps.  Matching
// lanes are counted together; no two warps share a counter.
__device__ __forceinline__ void warp_range(int n, int warp, int& c0, int& c1) {
    const int steps = (n + 31) / 32;
    c0 = (int)((long long)warp * steps / kRouteWarps) * 32;
    c1 = min(n, (int)((long long)(warp + 1) * steps / kRouteWarps) * 32);
}
__device__ __forceinline__ void count_slots(const int* ids, int n, int E, int* hist, int warp, int lane) {
    int* h = hist + warp * E;
    for (int e = lane; e < E; e += 32) h[e] = 0;
    __syncwarp();
    int c0, c1;
    warp_range(n, warp, c0, c1);
    for (int i = c0; i < c1; i += 32) {
        const int id = i + lane < c1 ? ids[i + lane] : -1;
        const unsigned same = __match_any_sync(0xffffffffu, id);
        if (id >= 0 && lane == __ffs(same) - 1) h[id] += __popc(same);
        __syncwarp();
    }
}
// After the rows of hist hold each warp's first position per expert: the slots to their places.
__device__ __forceinline__ void place_slots(const int* ids, int n, int E, int* hist, long long slot0, int* order, int warp, int lane) {
    int* h = hist + warp * E;
    int c0, c1;
    warp_range(n, warp, c0, c1);
    for (int i = c0; i < c1; i += 32) {
        const int id = i + lane < c1 ? ids[i + lane] : -1;
        const unsigned same = __match_any_sync(0xffffffffu, id);
        const int at = id >= 0 ? h[id] : 0;
        __syncwarp();
        if (id >= 0) {
            order[at + __popc(same & ((1u << lane) - 1u))] = (int)(slot0 + i + lane);
            if (lane == __ffs(same) - 1) h[id] = at + __popc(same);
        }
        __syncwarp();
    }
}

template <int EPL>
__global__ void __launch_bounds__(kRouteThreads) moe_route_kernel(const RouteParams p) {
    extern __shared__ __align__(16) int sm[];  // [kRouteWarps][E] picks, then counters; [E] totals
    __shared__ int tmp[kRouteWarps];
    const RouteCall& c = p.c;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    grid_dep_launch();
    grid_dep_wait();
    const int t0 = blockIdx.x * p.tile, t1 = min(c.T, t0 + p.tile);
    for (int t = t0 + warp; t < t1; t += kRouteWarps) route_token<EPL>(c, t, reinterpret_cast<float*>(sm) + warp * c.E, lane);
    if (!c.order) return;
    __syncthreads();  // the ids of this block's tokens are written
    const int n = (t1 - t0) * c.top_k;
    const int* ids = c.ids + (long long)t0 * c.top_k;
    count_slots(ids, n, c.E, sm, warp, lane);
    __syncthreads();
    int* tot = sm + kRouteWarps * c.E;
    for (int e = tid; e < c.E; e += kRouteThreads) {
        int v = 0;
#pragma unroll
        for (int w = 0; w < kRouteWarps; ++w) {
            const int u = sm[w * c.E + e];
            sm[w * c.E + e] = v;
            v += u;
        }
        tot[e] = v;
        if (p.blocks > 1) p.counts[(long long)blockIdx.x * c.E + e] = (unsigned)v;
    }
    if (p.blocks > 1) return;
    __syncthreads();
    const int all = block_scan(tot, c.E, tmp, tid);
    for (int e = tid; e < c.E; e += kRouteThreads) {
        c.offsets[e] = tot[e];
#pragma unroll
        for (int w = 0; w < kRouteWarps; ++w) sm[w * c.E + e] += tot[e];
    }
    if (tid == 0) c.offsets[c.E] = all;
    __syncthreads();
    place_slots(ids, n, c.E, sm, 0, c.order, warp, lane);
}

__global__ void __launch_bounds__(kRouteThreads) moe_order_kernel(const RouteParams p) {
    extern __shared__ __align__(16) int sm[];
    __shared__ int tmp[kRouteWarps];
    const RouteCall& c = p.c;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int t0 = blockIdx.x * p.tile, t1 = min(c.T, t0 + p.tile);
    const int n = (t1 - t0) * c.top_k;
    const int* ids = c.ids + (long long)t0 * c.top_k;
    grid_dep_launch();
    grid_dep_wait();
    // slots of expert e in the blocks before this one, and in all
    int* tot = sm + kRouteWarps * c.E;
    int before = 0, all = 0;
    if (tid < c.E)
        for (int b = 0; b < p.blocks; ++b) {
            const int v = (int)__ldcg(p.counts + (long long)b * c.E + tid);
            before += b < (int)blockIdx.x ? v : 0;
            all += v;
        }
    if (tid < c.E) tot[tid] = all;
    count_slots(ids, n, c.E, sm, warp, lane);
    __syncthreads();
    const int every = block_scan(tot, c.E, tmp, tid);
    if (tid < c.E) {
        if (blockIdx.x == 0) c.offsets[tid] = tot[tid];
        int v = tot[tid] + before;
#pragma unroll
        for (int w = 0; w < kRouteWarps; ++w) {
            const int u = sm[w * c.E + tid];
            sm[w * c.E + tid] = v;
            v += u;
        }
    }
    if (blockIdx.x == 0 && tid == 0) c.offsets[c.E] = every;
    __syncthreads();
    place_slots(ids, n, c.E, sm, (long long)t0 * c.top_k, c.order, warp, lane);
}

__global__ void moe_no_tokens_kernel(int* offsets, int E) {
    grid_dep_wait();
    for (int e = threadIdx.x; e <= E; e += blockDim.x) offsets[e] = 0;
}

// 32 tokens a block (two a warp) up to 256 blocks; the second launch reads
// every block's counts, so more blocks cost it more than they save
int route_tile(int T) { return T <= 32 * 256 ? 32 : (T + 255) / 256; }

}  // namespace

size_t route_workspace(int T, int E, int top_k) {
    const int tile = route_tile(T), blocks = (T + tile - 1) / tile;
    return blocks > 1 ? (size_t)blocks * E * 4 : 0;
}

cudaError_t launch_route(const RouteCall& c, void* ws, cudaStream_t s) {
    if (c.T == 0) {
        if (!c.offsets) return cudaSuccess;
        moe_no_tokens_kernel<<<1, 256, 0, s>>>(c.offsets, c.E);
        return cudaGetLastError();
    }
    RouteParams p;
    p.c = c;
    p.tile = route_tile(c.T);
    p.blocks = (c.T + p.tile - 1) / p.tile;
    p.counts = static_cast<unsigned*>(ws);
    const size_t smem = (size_t)(kRouteWarps + 1) * c.E * 4;  // at most 34 KB
    const unsigned g = (unsigned)p.blocks;
    const int epl = (c.E + 31) / 32;
    cudaError_t e = epl <= 1   ? launch_pdl(moe_route_kernel<1>, g, kRouteThreads, smem, s, p)
                    : epl <= 2 ? launch_pdl(moe_route_kernel<2>, g, kRouteThreads, smem, s, p)
                    : epl <= 4 ? launch_pdl(moe_route_kernel<4>, g, kRouteThreads, smem, s, p)
                    : epl <= 8 ? launch_pdl(moe_route_kernel<8>, g, kRouteThreads, smem, s, p)
                               : launch_pdl(moe_route_kernel<16>, g, kRouteThreads, smem, s, p);
    if (e != cudaSuccess || !c.order || p.blocks == 1) return e;
    return launch_pdl(moe_order_kernel, g, kRouteThreads, smem, s, p);
}

}  // namespace qmm
