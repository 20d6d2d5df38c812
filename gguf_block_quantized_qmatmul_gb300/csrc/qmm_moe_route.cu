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
// The order (a stable counting sort of the T k slots by expert) hands out no
// place by an atomic, so it is the same on every run: each block counts its tokens'
// slots by expert; in the second launch a block adds up the counts of all
// blocks (its own base positions and the offsets), and its warps rank their
// 32 consecutive slots at a time by matching lanes.  A call that fits one
// block does all of it in the first launch.
#include "qmm_q4g_internal.h"

namespace qmm {
namespace {

constexpr int kRouteTile = 32;  // tokens per block, up to 256 blocks
constexpr int kRouteMaxBlocks = 256;
// a warp per token of the tile, unless the picks of over 256 experts take too many registers
__host__ __device__ constexpr int route_warps(int epl) { return epl <= 8 ? 32 : 16; }


struct RouteParams {
    RouteCall c;
    int tile;      // tokens per block
    int blocks;
    unsigned group_magic;  // 2^22 / (experts per group), rounded up: e / group size for e < 512
    unsigned* counts;  // [blocks][E] slots of each block by expert (more than one block)
};

// order-preserving integer key of a float; -0 counts as +0, NaN ranks below -inf; 0 is "none"
__device__ __forceinline__ uint32_t pick_key(float f) {
    if (f != f) return 1u;
    const uint32_t u = __float_as_uint(f + 0.0f);
    return u & 0x80000000u ? ~u : u | 0x80000000u;
}

// One token: EPL experts per lane.  sk: the warp's row of picks in shared memory (with groups).
// Lane j < top_k returns choice j.
template <int EPL>
__device__ __forceinline__ int route_token(const RouteParams& p, long long tok, uint32_t* sk, int lane) {
    const RouteCall& c = p.c;
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
            if (e < c.E && !((kept >> ((e * p.group_magic) >> 22)) & 1u)) key[i] = 0u;
        }
    }
    // the k largest: lane j ends up with choice j; a lane looks for its own largest again
    // only after it gave it away
    int my_id = 0;
    float my_score = 0.0f, sum = 0.0f;
    uint32_t b = 0u;
    int bi = 0;
    auto local = [&]() {
        b = 0u;
        bi = 0;
#pragma unroll
        for (int i = 0; i < EPL; ++i) {
            const bool more = key[i] > b;
            b = more ? key[i] : b;
            bi = more ? i : bi;
        }
    };
    local();
    for (int j = 0; j < c.top_k; ++j) {
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
        if (lane == (int)(id & 31u)) local();
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
    return my_id;
}

// exclusive prefix sum of a[0..n) in shared memory by the whole block, n <= 512; returns the total
template <int W>
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
    for (int i = 0; i < W; ++i) {
        const int u = tmp[i];
        if (i < warp) before += u;
        all += u;
    }
    if (tid < n) a[tid] = before + incl - v;
    __syncthreads();
    return all;
}

// Counts n ids by expert, a row of `hist` [W][E] per warp; each warp has a
// consecutive part of the 32-slot steps.  Matching lanes are counted together;
// no two warps share a counter.
template <int W>
__device__ __forceinline__ void warp_range(int n, int warp, int& c0, int& c1) {
    const int steps = (n + 31) / 32;
    c0 = (int)((long long)warp * steps / W) * 32;
    c1 = min(n, (int)((long long)(warp + 1) * steps / W) * 32);
}
template <int W>
__device__ __forceinline__ void count_slots(const int* ids, int n, int E, int* hist, int warp, int lane) {
    int* h = hist + warp * E;
    for (int e = lane; e < E; e += 32) h[e] = 0;
    __syncwarp();
    int c0, c1;
    warp_range<W>(n, warp, c0, c1);
    for (int i = c0; i < c1; i += 32) {
        const int id = i + lane < c1 ? ids[i + lane] : -1;
        const unsigned same = __match_any_sync(0xffffffffu, id);
        if (id >= 0 && lane == __ffs(same) - 1) h[id] += __popc(same);
        __syncwarp();
    }
}
// After the rows of hist hold each warp's first position per expert: the slots to their places.
template <int W>
__device__ __forceinline__ void place_slots(const int* ids, int n, int E, int* hist, long long slot0, int* order, int warp, int lane) {
    int* h = hist + warp * E;
    int c0, c1;
    warp_range<W>(n, warp, c0, c1);
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

// One token: one warp does it all, with no barrier.
template <int EPL>
__global__ void __launch_bounds__(32) moe_route_one_kernel(const RouteParams p) {
    extern __shared__ __align__(16) uint32_t sk[];
    const RouteCall& c = p.c;
    const int lane = threadIdx.x;
    grid_dep_launch();
    grid_dep_wait();
    const int id = route_token<EPL>(p, 0, sk, lane);
    if (!c.order) return;
    int rank = 0, below[EPL];  // slots of lower experts than lane + 32 i (a token's experts differ)
#pragma unroll
    for (int i = 0; i < EPL; ++i) below[i] = 0;
    for (int j = 0; j < c.top_k; ++j) {
        const int other = __shfl_sync(0xffffffffu, id, j);
        rank += other < id;
#pragma unroll
        for (int i = 0; i < EPL; ++i) below[i] += other < lane + 32 * i;
    }
    if (lane < c.top_k) c.order[rank] = lane;
#pragma unroll
    for (int i = 0; i < EPL; ++i)
        if (lane + 32 * i < c.E) c.offsets[lane + 32 * i] = below[i];
    if (lane == 0) c.offsets[c.E] = c.top_k;
}

template <int EPL>
__global__ void __launch_bounds__(route_warps(EPL) * 32) moe_route_kernel(const RouteParams p) {
    extern __shared__ __align__(16) int sm[];  // [W][E] picks, then counters; [E] totals
    constexpr int W = route_warps(EPL), kThreads = W * 32;
    __shared__ int tmp[W];
    const RouteCall& c = p.c;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    grid_dep_launch();
    grid_dep_wait();
    const int t0 = blockIdx.x * p.tile, t1 = min(c.T, t0 + p.tile);
    for (int t = t0 + warp; t < t1; t += W) route_token<EPL>(p, t, reinterpret_cast<uint32_t*>(sm) + warp * c.E, lane);
    if (!c.order) return;
    __syncthreads();  // the ids of this block's tokens are written
    const int n = (t1 - t0) * c.top_k;
    const int* ids = c.ids + (long long)t0 * c.top_k;
    count_slots<W>(ids, n, c.E, sm, warp, lane);
    __syncthreads();
    int* tot = sm + W * c.E;
    for (int e = tid; e < c.E; e += kThreads) {
        int v = 0;
#pragma unroll
        for (int w = 0; w < W; ++w) {
            const int u = sm[w * c.E + e];
            sm[w * c.E + e] = v;
            v += u;
        }
        tot[e] = v;
        if (p.blocks > 1) p.counts[(long long)blockIdx.x * c.E + e] = (unsigned)v;
    }
    if (p.blocks > 1) return;
    __syncthreads();
    const int all = block_scan<W>(tot, c.E, tmp, tid);
    for (int e = tid; e < c.E; e += kThreads) {
        c.offsets[e] = tot[e];
#pragma unroll
        for (int w = 0; w < W; ++w) sm[w * c.E + e] += tot[e];
    }
    if (tid == 0) c.offsets[c.E] = all;
    __syncthreads();
    place_slots<W>(ids, n, c.E, sm, 0, c.order, warp, lane);
}

constexpr int kOrderWarps = 16, kOrderThreads = kOrderWarps * 32;
__global__ void __launch_bounds__(kOrderThreads) moe_order_kernel(const RouteParams p) {
    extern __shared__ __align__(16) int sm[];  // [W][E] counters; [E] totals; [E] slots in earlier blocks
    __shared__ int tmp[kOrderWarps];
    const RouteCall& c = p.c;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, E = c.E;
    const int t0 = blockIdx.x * p.tile, t1 = min(c.T, t0 + p.tile);
    const int n = (t1 - t0) * c.top_k;
    const int* ids = c.ids + (long long)t0 * c.top_k;
    grid_dep_launch();
    int* tot = sm + kOrderWarps * E;
    int* pre = tot + E;
    for (int e = tid; e < 2 * E; e += kOrderThreads) tot[e] = 0;
    __syncthreads();
    grid_dep_wait();
    // slots of every expert in all blocks and in those before this one: a warp adds up every
    // sixteenth block's counts, eight rows in flight (integer sums: their order does not matter)
    for (int e = lane; e < E; e += 32) {
        int before = 0, all = 0;
        for (int b0 = warp; b0 < p.blocks; b0 += 8 * kOrderWarps) {
            int v[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const int b = b0 + i * kOrderWarps;
                v[i] = b < p.blocks ? (int)__ldcg(p.counts + (long long)b * E + e) : 0;
            }
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                before += b0 + i * kOrderWarps < (int)blockIdx.x ? v[i] : 0;
                all += v[i];
            }
        }
        atomicAdd(&tot[e], all);
        atomicAdd(&pre[e], before);
    }
    count_slots<kOrderWarps>(ids, n, E, sm, warp, lane);
    __syncthreads();
    const int every = block_scan<kOrderWarps>(tot, E, tmp, tid);
    for (int e = tid; e < E; e += kOrderThreads) {
        if (blockIdx.x == 0) c.offsets[e] = tot[e];
        int v = tot[e] + pre[e];
#pragma unroll
        for (int w = 0; w < kOrderWarps; ++w) {
            const int u = sm[w * E + e];
            sm[w * E + e] = v;
            v += u;
        }
    }
    if (blockIdx.x == 0 && tid == 0) c.offsets[E] = every;
    __syncthreads();
    place_slots<kOrderWarps>(ids, n, E, sm, (long long)t0 * c.top_k, c.order, warp, lane);
}

__global__ void moe_no_tokens_kernel(int* offsets, int E) {
    grid_dep_wait();
    for (int e = threadIdx.x; e <= E; e += blockDim.x) offsets[e] = 0;
}

// the second launch reads every block's counts, so that more blocks would cost it more than they save
int route_tile(int T) { return T <= kRouteTile * kRouteMaxBlocks ? kRouteTile : (T + kRouteMaxBlocks - 1) / kRouteMaxBlocks; }

template <int EPL>
cudaError_t route_go(const RouteParams& p, cudaStream_t s) {
    if (p.c.T == 1) return launch_pdl(moe_route_one_kernel<EPL>, 1u, 32u, (size_t)p.c.E * 4, s, p);
    const size_t smem = (size_t)(route_warps(EPL) + 1) * p.c.E * 4;  // at most 35 KB
    return launch_pdl(moe_route_kernel<EPL>, (unsigned)p.blocks, (unsigned)(route_warps(EPL) * 32), smem, s, p);
}

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
    const int gs = c.E / c.groups;
    p.group_magic = ((1u << 22) + gs - 1) / gs;
    const int epl = (c.E + 31) / 32;
    const cudaError_t e = epl <= 1   ? route_go<1>(p, s)
                          : epl <= 2 ? route_go<2>(p, s)
                          : epl <= 4 ? route_go<4>(p, s)
                          : epl <= 8 ? route_go<8>(p, s)
                                     : route_go<16>(p, s);
    if (e != cudaSuccess || !c.order || p.blocks == 1) return e;
    return launch_pdl(moe_order_kernel, (unsigned)p.blocks, kOrderThreads, (size_t)(kOrderWarps + 2) * c.E * 4, s, p);
}

}  // namespace qmm
