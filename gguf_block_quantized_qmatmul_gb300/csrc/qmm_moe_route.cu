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
// its picks in registers, consecutive experts a lane, and every lane knows its
// largest; a selection step is one warp-wide integer reduction (redux) of
// those on order-preserving keys and a ballot, whose lowest lane has the
// lowest expert of equals and looks for its next largest.
//
// The order (a stable counting sort of the T k slots by expert) hands out no
// place by an atomic, so it is the same on every run.  A tile is up to 32
// tokens, and a token's experts differ, so a tile's slots of an expert are a
// 32-bit mask over its tokens: its population count is the tile's number of
// them (a byte), and that of its lower bits a slot's rank.  The first launch
// writes every tile's counts; in the second a block adds up those of all tiles
// (its own first positions and the offsets) and places the slots of its tiles.
// A call of one tile does all of it in the first launch.
//
// Measured: 4096 tokens, 256 experts in 8 groups, top 8, sigmoid with bias, bf16:
// 16 us with the order (its bytes take 0.4; the selection's 5.3 million warp
// instructions are 8 of them, the second launch with the counts' sums the rest);
// one token of 64 experts 2.1 us, a launch.
#include "qmm_q4g_internal.h"

namespace qmm {
namespace {

constexpr int kRouteTile = 32;   // tokens per tile, at most: one bit each
constexpr int kOrderTiles = 32;  // tiles that an order block places at a time
// a warp per token of the tile, unless the picks of over 256 experts take too many registers
__host__ __device__ constexpr int route_warps(int epl) { return epl <= 8 ? 32 : 16; }

struct RouteParams {
    RouteCall c;
    int tile;              // tokens per tile (a block of the first launch)
    int blocks;            // tiles
    uint8_t* counts;       // [tiles][stride]: slots of each tile by expert (more than one tile)
    int stride;            // bytes from a tile's counts to the next: E rounded up to 16
    int per;               // tiles per block of the second launch
    int vec, vec_bias;     // logits, bias: a lane's experts may be read as vectors
    int group_lanes_log2;  // a group is 2^this lanes' experts; -1: it is not
    unsigned group_magic;  // 2^22 / (experts per group), rounded up: e / group size for e < 512
};

// order-preserving integer key of a float; -0 counts as +0, NaN ranks below -inf; 0 is "none"
__device__ __forceinline__ uint32_t pick_key(float f) {
    if (f != f) return 1u;
    const uint32_t u = __float_as_uint(f + 0.0f);
    return u & 0x80000000u ? ~u : u | 0x80000000u;
}

// EPL consecutive values of 4-byte words or fewer, as raw words; vec: they may be read 16 (8, 4) bytes at a time
template <int WORDS>
__device__ __forceinline__ void load_words(const uint32_t* p, uint32_t w[WORDS]) {
    if constexpr (WORDS % 4 == 0) {
#pragma unroll
        for (int i = 0; i < WORDS / 4; ++i) {
            const uint4 v = reinterpret_cast<const uint4*>(p)[i];
            w[4 * i] = v.x;
            w[4 * i + 1] = v.y;
            w[4 * i + 2] = v.z;
            w[4 * i + 3] = v.w;
        }
    } else if constexpr (WORDS == 2) {
        const uint2 v = *reinterpret_cast<const uint2*>(p);
        w[0] = v.x;
        w[1] = v.y;
    } else {
        w[0] = *p;
    }
}

// One token: EPL consecutive experts per lane.  sk: the warp's row of picks in
// shared memory (groups that are not whole powers of two of lanes).  Lane j <
// top_k returns choice j.
template <int EPL>
__device__ __forceinline__ int route_token(const RouteParams& p, long long tok, uint32_t* sk, int lane) {
    const RouteCall& c = p.c;
    float score[EPL];
    uint32_t key[EPL];
    const long long base = tok * c.ldl;
    const int e0 = lane * EPL;
    float m = -INFINITY;
    // the type is told apart outside of the loads, so that they are in flight together
    if (p.vec) {  // E is a multiple of EPL: a lane has all of its experts or none
        if (c.xt == X_F32) {
            uint32_t w[EPL];
            if (e0 < c.E) load_words<EPL>(reinterpret_cast<const uint32_t*>(static_cast<const float*>(c.logits) + base + e0), w);
#pragma unroll
            for (int i = 0; i < EPL; ++i) score[i] = e0 < c.E ? __uint_as_float(w[i]) : -INFINITY;
        } else if constexpr (EPL >= 2) {
            uint32_t w[EPL / 2];
            if (e0 < c.E) load_words<EPL / 2>(reinterpret_cast<const uint32_t*>(static_cast<const uint16_t*>(c.logits) + base + e0), w);
#pragma unroll
            for (int i = 0; i < EPL; ++i) {
                const uint32_t h = i & 1 ? w[i / 2] >> 16 : w[i / 2] & 0xffffu;
                score[i] = e0 >= c.E ? -INFINITY : c.xt == X_F16 ? h2f(h) : __uint_as_float(h << 16);
            }
        }
    } else if (c.xt == X_F32) {
#pragma unroll
        for (int i = 0; i < EPL; ++i) score[i] = e0 + i < c.E ? static_cast<const float*>(c.logits)[base + e0 + i] : -INFINITY;
    } else {
        uint16_t raw[EPL];
#pragma unroll
        for (int i = 0; i < EPL; ++i) raw[i] = e0 + i < c.E ? static_cast<const uint16_t*>(c.logits)[base + e0 + i] : (uint16_t)0;
#pragma unroll
        for (int i = 0; i < EPL; ++i)
            score[i] = e0 + i >= c.E ? -INFINITY : c.xt == X_F16 ? h2f(raw[i]) : __uint_as_float((uint32_t)raw[i] << 16);
    }
#pragma unroll
    for (int i = 0; i < EPL; ++i) {
        if (score[i] != score[i]) score[i] = -INFINITY;  // a NaN logit is a masked one
        m = fmaxf(m, score[i]);
    }
    if (!c.sigmoid) {
        float total = 0.0f;
#pragma unroll
        for (int o = 16; o; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
#pragma unroll
        for (int i = 0; i < EPL; ++i) {
            const float l = score[i];
            // a row whose mask leaves nothing has no scores; l = m also covers +inf
            const float s = m == -INFINITY ? 0.0f : l == m ? 1.0f : expf(l - m);
            if (!c.bias) key[i] = pick_key(l);
            score[i] = e0 + i < c.E ? s : 0.0f;
            total += score[i];
        }
        if (c.bias || !c.renorm) {
#pragma unroll
            for (int o = 16; o; o >>= 1) total += __shfl_xor_sync(0xffffffffu, total, o);
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
        float b[EPL];
        if (p.vec_bias && e0 < c.E) {
            uint32_t w[EPL];
            load_words<EPL>(reinterpret_cast<const uint32_t*>(c.bias + e0), w);
#pragma unroll
            for (int i = 0; i < EPL; ++i) b[i] = __uint_as_float(w[i]);
        } else {
#pragma unroll
            for (int i = 0; i < EPL; ++i) b[i] = e0 + i < c.E ? __ldg(c.bias + e0 + i) : 0.0f;
        }
#pragma unroll
        for (int i = 0; i < EPL; ++i) key[i] = pick_key(score[i] + b[i]);
    }
#pragma unroll
    for (int i = 0; i < EPL; ++i)
        if (e0 + i >= c.E) key[i] = 0u;
    if (c.groups > 1) {
        uint32_t b1 = 0u, b2 = 0u;  // the two largest picks of this lane's group, in the group's first lane
        int log_lanes;              // lanes per group, a power of two
        if (p.group_lanes_log2 >= 0) {  // a group is whole lanes
            log_lanes = p.group_lanes_log2;
#pragma unroll
            for (int i = 0; i < EPL; ++i) {
                b2 = max(b2, min(b1, key[i]));
                b1 = max(b1, key[i]);
            }
        } else {  // through shared memory: lane r of a group takes its picks r, r + lanes, ...
            const int gs = c.E / c.groups;
            log_lanes = 5;
            while ((c.groups << log_lanes) > 32) --log_lanes;
            __syncwarp();
#pragma unroll
            for (int i = 0; i < EPL; ++i)
                if (e0 + i < c.E) sk[e0 + i] = key[i];
            __syncwarp();
            const int q = lane >> log_lanes;
            if (q < c.groups)
                for (int r = lane & ((1 << log_lanes) - 1); r < gs; r += 1 << log_lanes) {
                    const uint32_t k = sk[q * gs + r];
                    b2 = max(b2, min(b1, k));
                    b1 = max(b1, k);
                }
        }
        for (int o = (1 << log_lanes) >> 1; o; o >>= 1) {
            const uint32_t o1 = __shfl_xor_sync(0xffffffffu, b1, o), o2 = __shfl_xor_sync(0xffffffffu, b2, o);
            b2 = max(max(b2, o2), min(b1, o1));
            b1 = max(b1, o1);
        }
        uint32_t gk = b1;
        if (c.top2 && b2 != 0u) {
            const uint32_t u1 = b1 & 0x80000000u ? b1 & 0x7fffffffu : ~b1, u2 = b2 & 0x80000000u ? b2 & 0x7fffffffu : ~b2;
            gk = pick_key(__uint_as_float(u1) + __uint_as_float(u2));
        }
        if ((lane >> log_lanes) >= c.groups || (lane & ((1 << log_lanes) - 1)) != 0) gk = 0u;
        uint32_t kept = 0u;  // bit per group
        for (int s = 0; s < c.top_groups; ++s) {
            const uint32_t best = __reduce_max_sync(0xffffffffu, gk);
            const int l0 = __ffs(__ballot_sync(0xffffffffu, gk == best)) - 1;
            kept |= 1u << (l0 >> log_lanes);
            if (lane == l0) gk = 0u;
        }
        if (p.group_lanes_log2 >= 0) {
            if (!((kept >> (lane >> log_lanes)) & 1u))
#pragma unroll
                for (int i = 0; i < EPL; ++i) key[i] = 0u;
        } else {
#pragma unroll
            for (int i = 0; i < EPL; ++i)
                if (e0 + i < c.E && !((kept >> (((unsigned)(e0 + i) * p.group_magic) >> 22)) & 1u)) key[i] = 0u;
        }
    }
    // the k largest: lane j ends up with choice j; a lane looks for its own largest again
    // only after it gave it away (the lowest lane of equals has the lowest expert)
    int my_id = 0;
    float my_score = 0.0f, sum = 0.0f;
    uint32_t b = 0u;
    int bi = 0;
    float bs = 0.0f;
    auto local = [&]() {
        b = 0u;
        bi = 0;
        bs = 0.0f;
#pragma unroll
        for (int i = 0; i < EPL; ++i) {
            const bool more = key[i] > b;
            b = more ? key[i] : b;
            bi = more ? i : bi;
            bs = more ? score[i] : bs;
        }
    };
    local();
    for (int j = 0; j < c.top_k; ++j) {
        const uint32_t best = __reduce_max_sync(0xffffffffu, b);
        const int l0 = __ffs(__ballot_sync(0xffffffffu, b == best)) - 1;
        const int id = __shfl_sync(0xffffffffu, e0 + bi, l0);
        const float s = __shfl_sync(0xffffffffu, bs, l0);
        if (lane == l0) {
#pragma unroll
            for (int i = 0; i < EPL; ++i) key[i] = i == bi ? 0u : key[i];
            local();
        }
        sum += s;
        if (lane == j) {
            my_id = id;
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
    int rank = 0, below[EPL];  // slots of lower experts than this lane's i-th (a token's experts differ)
#pragma unroll
    for (int i = 0; i < EPL; ++i) below[i] = 0;
    for (int j = 0; j < c.top_k; ++j) {
        const int other = __shfl_sync(0xffffffffu, id, j);
        rank += other < id;
#pragma unroll
        for (int i = 0; i < EPL; ++i) below[i] += other < lane * EPL + i;
    }
    if (lane < c.top_k) c.order[rank] = lane;
#pragma unroll
    for (int i = 0; i < EPL; ++i)
        if (lane * EPL + i < c.E) c.offsets[lane * EPL + i] = below[i];
    if (lane == 0) c.offsets[c.E] = c.top_k;
}

template <int EPL>
__global__ void __launch_bounds__(route_warps(EPL) * 32) moe_route_kernel(const RouteParams p) {
    extern __shared__ __align__(16) uint32_t sm[];  // [E] masks; [E] totals; [W][E] picks (groups that are not whole lanes)
    constexpr int W = route_warps(EPL), kThreads = W * 32;
    __shared__ int tmp[W];
    const RouteCall& c = p.c;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    uint32_t* mask = sm;
    if (c.order) {
        for (int e = tid; e < c.E; e += kThreads) mask[e] = 0u;
        __syncthreads();
    }
    grid_dep_launch();
    grid_dep_wait();
    const int t0 = blockIdx.x * p.tile, t1 = min(c.T, t0 + p.tile);
    int id[(kRouteTile + W - 1) / W];  // lane j: choice j of this warp's tokens
#pragma unroll
    for (int i = 0; i < (kRouteTile + W - 1) / W; ++i) {
        const int t = t0 + warp + i * W;
        id[i] = -1;
        if (t >= t1) continue;
        const int got = route_token<EPL>(p, t, sm + (2 + warp) * c.E, lane);
        if (lane < c.top_k) id[i] = got;
        if (c.order && lane < c.top_k) atomicOr(&mask[got], 1u << (t - t0));
    }
    if (!c.order) return;
    __syncthreads();
    if (p.blocks > 1) {
        for (int e = tid; e < c.E; e += kThreads) p.counts[(long long)blockIdx.x * p.stride + e] = (uint8_t)__popc(mask[e]);
        return;
    }
    int* tot = reinterpret_cast<int*>(sm + c.E);
    for (int e = tid; e < c.E; e += kThreads) tot[e] = __popc(mask[e]);
    __syncthreads();
    const int all = block_scan<W>(tot, c.E, tmp, tid);
    for (int e = tid; e < c.E; e += kThreads) c.offsets[e] = tot[e];
    if (tid == 0) c.offsets[c.E] = all;
#pragma unroll
    for (int i = 0; i < (kRouteTile + W - 1) / W; ++i) {
        const int t = warp + i * W;
        if (id[i] >= 0) c.order[tot[id[i]] + __popc(mask[id[i]] & ((1u << t) - 1u))] = t * c.top_k + lane;
    }
}

constexpr int kOrderWarps = 16, kOrderThreads = kOrderWarps * 32;
constexpr int kOrderRows = 1000 * 2 * kOrderWarps;
__global__ void __launch_bounds__(kOrderThreads) moe_order_kernel(const RouteParams p) {
    // [held][E] masks; [E] totals, then first positions; [E] slots in earlier tiles; [2][W][stride / 2] sums
    extern __shared__ __align__(16) uint32_t sm[];
    __shared__ int tmp[kOrderWarps];
    const RouteCall& c = p.c;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, E = c.E;
    const int b0 = blockIdx.x * p.per, b1 = min(p.blocks, b0 + p.per);
    grid_dep_launch();
    const int held = min(p.per, kOrderTiles);
    uint32_t* sums = sm;  // first, as it is written 16 bytes at a time
    const int words = p.stride / 2;
    uint32_t* mask = sums + 2 * kOrderWarps * words;
    int* tot = reinterpret_cast<int*>(mask + held * E);
    int* pre = tot + E;
    for (int e = tid; e < (held + 2) * E; e += kOrderThreads) mask[e] = 0u;
    grid_dep_wait();
    // Slots of every expert in the tiles before this block's and in the rest.  A half warp reads
    // a tile's counts of 256 experts, 16 a lane, four tiles in flight; bytes are added up in 16-bit
    // halves (at most 1000 of up to 32 in either half warp), then the warps' sums.
    for (int base = 0; base < p.blocks; base += kOrderRows) {
        const int end = min(p.blocks, base + kOrderRows);
        for (int c0 = 0; c0 < p.stride; c0 += 256)
            for (int half = 0; half < 2; ++half) {
                // The half warps' trip counts differ, and nothing brings them together after the loop
                // but the shuffle itself: every lane takes part in it, those without experts too.
                const int e0 = c0 + 16 * (lane & 15);
                const bool on = e0 < p.stride;
                const int from = half ? max(base, min(b0, end)) : base, to = !on ? from : half ? end : min(b0, end);
                uint32_t s8[8] = {};
                for (int b = from + 2 * warp + (lane >> 4); b < to; b += 8 * kOrderWarps) {
                    uint4 v[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const int bb = b + i * 2 * kOrderWarps;
                        v[i] = bb < to ? __ldcg(reinterpret_cast<const uint4*>(p.counts + (long long)bb * p.stride + e0)) : make_uint4(0u, 0u, 0u, 0u);
                    }
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const uint32_t u[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
#pragma unroll
                        for (int q = 0; q < 4; ++q) {
                            s8[q] += u[q] & 0x00ff00ffu;             // experts 4 q, 4 q + 2
                            s8[4 + q] += (u[q] >> 8) & 0x00ff00ffu;  // 4 q + 1, 4 q + 3
                        }
                    }
                }
#pragma unroll
                for (int q = 0; q < 8; ++q) s8[q] += __shfl_xor_sync(0xffffffffu, s8[q], 16);
                if (on && lane < 16) {
                    uint4* to4 = reinterpret_cast<uint4*>(sums + (half * kOrderWarps + warp) * words + e0 / 2);
                    to4[0] = make_uint4(s8[0], s8[1], s8[2], s8[3]);
                    to4[1] = make_uint4(s8[4], s8[5], s8[6], s8[7]);
                }
            }
        __syncthreads();
        for (int e = tid; e < E; e += kOrderThreads) {
            const int r = e & 15, word = (e >> 4) * 8 + (r & 1) * 4 + (r >> 2), sh = r & 2 ? 16 : 0;
            int v = 0, u = 0;
#pragma unroll
            for (int w = 0; w < kOrderWarps; ++w) {
                v += (int)((sums[w * words + word] >> sh) & 0xffffu);
                u += (int)((sums[(kOrderWarps + w) * words + word] >> sh) & 0xffffu);
            }
            pre[e] += v;
            tot[e] += v + u;
        }
        __syncthreads();
    }
    const int every = block_scan<kOrderWarps>(tot, E, tmp, tid);
    if (blockIdx.x == 0) {
        for (int e = tid; e < E; e += kOrderThreads) c.offsets[e] = tot[e];
        if (tid == 0) c.offsets[E] = every;
    }
    for (int c0 = b0; c0 < b1; c0 += kOrderTiles) {
        // masks of these tiles from their ids, then each tile's first positions in the masks' place
        const int tiles = min(kOrderTiles, b1 - c0);
        const long long s0 = (long long)c0 * p.tile * c.top_k;
        const int n = (min(c.T, (c0 + tiles) * p.tile) - c0 * p.tile) * c.top_k;
        if (c0 > b0) {
            __syncthreads();
            for (int e = tid; e < held * E; e += kOrderThreads) mask[e] = 0u;
            __syncthreads();
        }
        for (int i = tid; i < n; i += kOrderThreads) {
            const int tok = i / c.top_k, tl = tok / p.tile;
            atomicOr(&mask[tl * E + c.ids[s0 + i]], 1u << (tok - tl * p.tile));
        }
        __syncthreads();
        for (int i = tid; i < n; i += kOrderThreads) {
            const int tok = i / c.top_k, tl = tok / p.tile, id = c.ids[s0 + i];
            int at = tot[id] + pre[id] + __popc(mask[tl * E + id] & ((1u << (tok - tl * p.tile)) - 1u));
            for (int u = 0; u < tl; ++u) at += __popc(mask[u * E + id]);
            c.order[at] = (int)(s0 + i);
        }
        if (c0 + kOrderTiles < b1) {  // more tiles follow
            __syncthreads();
            for (int e = tid; e < E; e += kOrderThreads) {
                int v = 0;
                for (int u = 0; u < tiles; ++u) v += __popc(mask[u * E + e]);
                pre[e] += v;
            }
        }
    }
}

__global__ void moe_no_tokens_kernel(int* offsets, int E) {
    grid_dep_wait();
    for (int e = threadIdx.x; e <= E; e += blockDim.x) offsets[e] = 0;
}

// Tokens per tile: what gives every SM one block, 8 to 32 (a warp each)
int route_tile(int T, int sms) {
    const int even = (T + sms - 1) / sms;
    return T <= kRouteTile ? kRouteTile : even < 8 ? 8 : even < kRouteTile ? even : kRouteTile;
}
int sm_count() {
    int sms = 0, smem = 0;
    return device_constants(nullptr, &sms, &smem) == cudaSuccess && sms > 0 ? sms : 1;
}

template <int EPL>
cudaError_t route_go(const RouteParams& p, cudaStream_t s) {
    if (p.c.T == 1) return launch_pdl(moe_route_one_kernel<EPL>, 1u, 32u, (size_t)p.c.E * 4, s, p);
    const size_t smem = (size_t)(2 + (p.c.groups > 1 && p.group_lanes_log2 < 0 ? route_warps(EPL) : 0)) * p.c.E * 4;  // at most 37 KB
    return launch_pdl(moe_route_kernel<EPL>, (unsigned)p.blocks, (unsigned)(route_warps(EPL) * 32), smem, s, p);
}

}  // namespace

size_t route_workspace(int T, int E, int top_k) {
    const int tile = route_tile(T, sm_count()), blocks = (T + tile - 1) / tile;
    return blocks > 1 ? (size_t)blocks * ((E + 15) / 16 * 16) : 0;
}

cudaError_t launch_route(const RouteCall& c, void* ws, cudaStream_t s) {
    if (c.T == 0) {
        if (!c.offsets) return cudaSuccess;
        moe_no_tokens_kernel<<<1, 256, 0, s>>>(c.offsets, c.E);
        return cudaGetLastError();
    }
    RouteParams p;
    p.c = c;
    p.tile = route_tile(c.T, sm_count());
    p.stride = (c.E + 15) / 16 * 16;
    p.blocks = (c.T + p.tile - 1) / p.tile;
    p.counts = static_cast<uint8_t*>(ws);
    p.per = (p.blocks + 63) / 64;  // at most 64 order blocks: each reads all counts
    const int gs = c.E / c.groups;
    p.group_magic = ((1u << 22) + gs - 1) / gs;
    int epl = 1;  // experts per lane
    while (epl * 32 < c.E) epl *= 2;
    const int bytes = epl * x_size(c.xt), chunk = bytes < 16 ? bytes : 16;
    p.vec = bytes >= 4 && c.E % epl == 0 && (c.ldl * x_size(c.xt)) % chunk == 0 && (reinterpret_cast<uintptr_t>(c.logits) & (chunk - 1)) == 0;
    p.vec_bias = c.bias && c.E % epl == 0 && (reinterpret_cast<uintptr_t>(c.bias) & ((epl < 4 ? epl * 4 : 16) - 1)) == 0;
    p.group_lanes_log2 = -1;
    if (gs % epl == 0 && ((gs / epl) & (gs / epl - 1)) == 0)
        for (p.group_lanes_log2 = 0; (epl << p.group_lanes_log2) < gs;) ++p.group_lanes_log2;
    const cudaError_t e = epl <= 1   ? route_go<1>(p, s)
                          : epl <= 2 ? route_go<2>(p, s)
                          : epl <= 4 ? route_go<4>(p, s)
                          : epl <= 8 ? route_go<8>(p, s)
                                     : route_go<16>(p, s);
    if (e != cudaSuccess || !c.order || p.blocks == 1) return e;
    const int held = p.per < kOrderTiles ? p.per : kOrderTiles;
    static unsigned long long done = 0;
    const cudaError_t e2 = ensure_smem(moe_order_kernel, 112 * 1024, done);  // 102 KB for 512 experts and 32 tiles
    if (e2 != cudaSuccess) return e2;
    return launch_pdl(moe_order_kernel, (unsigned)((p.blocks + p.per - 1) / p.per), kOrderThreads, (size_t)((held + 2) * c.E + kOrderWarps * p.stride) * 4, s, p);
}

}  // namespace qmm
